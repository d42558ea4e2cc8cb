// Pieces shared by the 16-bit matrix products of the operators (grouped.hip, adapter.hip), gfx950 only:
// element types, LDS DMA through buffer descriptors, fragment reads, and the search for a work-group's tile.
//
// An operand tile holds 64 values of the contraction (one K step) for each of its rows or columns, in one
// of two LDS forms:
//   KC  (contraction contiguous in memory): one 128-byte LDS row per operand row, its eight 16-byte chunks
//       XOR-swizzled by row; a fragment is one ds_read_b128 per lane.
//   KS  (contraction strided: memory row = contraction index): one LDS row of W columns per contraction
//       index, its 32-byte pairs of chunks XOR-swizzled by row; a fragment is two ds_read_b64_tr_b16, which
//       transpose 4 x 16 blocks on the way to the registers.
// Both forms give lane l of a 16 x 32 fragment row (or column) l % 16 and contraction 8 * (l / 16) .. + 7,
// so an operand of one form pairs with one of the other.
//
// Every tile edge is handled by the buffer descriptor: a DMA lane whose offset is not below num_records
// writes zeros to LDS and reads no memory.  Rows past a group's end, contraction indices past its length and
// steps past the last one all become zeros in BOTH operands, so that a NaN behind the edge meets no sum.
#pragma once

#include "mm_internal.h"
#include "../../include/mega_moe_ops.h"

namespace mm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// Element types: the MFMA, and rounding (to nearest even) of two fp32 values into one word; kNarrow: fewer exponents
// than fp32.
struct Bf16 {
    static constexpr bool kNarrow = false;
    static __device__ __forceinline__ f32x4 mfma(i32x4 a, i32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2_t));
    }
    static __device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
};
struct Fp16 {
    static constexpr bool kNarrow = true;
    static __device__ __forceinline__ f32x4 mfma(i32x4 a, i32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, f16x2_t));
    }
    static __device__ __forceinline__ float low(uint32_t w) { return (float)__builtin_bit_cast(f16x2_t, w)[0]; }
    static __device__ __forceinline__ float high(uint32_t w) { return (float)__builtin_bit_cast(f16x2_t, w)[1]; }
};

constexpr int kStepK = 64;                   // contraction values per step: 128 bytes of a KC row
constexpr uint32_t kPastEnd = 0x80000000u;   // an offset that no descriptor here reaches (num_records < 2^31)

// ---------------------------------------------------------------- LDS DMA
__device__ __forceinline__ uint32_t lds_byte(const void* p) {
    return (uint32_t)(uintptr_t)(lds_void) const_cast<void*>(p);
}
__device__ __forceinline__ u32x4 buffer_of(const void* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    u32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);
    r[2] = __builtin_amdgcn_readfirstlane(bytes);
    r[3] = 0x00020000u;
    return r;
}
// 16 bytes per lane from descriptor + off to LDS at dst + lane * 16; zeros where off >= num_records.  Inline
// asm: the waits for these writes are placed by hand (wait_vm_barrier), since the compiler, which cannot tell
// the stages apart, would drain every DMA in flight before each LDS read.  An LDS DMA reads M0 no sooner than one wait
// state after its write; the compiler puts the s_nop between its own, and does not look into asm.
__device__ __forceinline__ void dma_rows(u32x4 desc, uint32_t off, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(off), "s"(desc), "s"(__builtin_amdgcn_readfirstlane(dst)) : "memory", "m0");
}
// At most N of this wave's vector-memory operations still outstanding and its LDS reads returned; then barrier.
template <int N>
__device__ __forceinline__ void wait_vm_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt immediate");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// KC: 16-byte chunk c of row r sits at position c ^ kc_swz(r).  A ds_read_b128 is served in four passes of 16
// lanes, each over all 64 banks: one pass takes eight rows of one lane group's chunk c and the other eight rows
// of its neighbour's, c ^ 1.  With r / 2 as the swizzle those 16 lanes meet 16 different 16-byte slots, whichever eight
// rows they are (r ^ (r / 8), which suits 16 lanes of one chunk, stalled half of the LDS-active cycles).  KS: 32-byte pair p of contraction row r sits at p ^ ks_swz(r); the eight
// rows {0..3, 8..11} (or {4..7, 12..15}) that half a wave reads at once get eight different 32-byte slots.
__device__ __forceinline__ int kc_swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int ks_swz(int r) { return (r & 3) | ((r >> 1) & 4); }

// The DMA of one KC operand tile of ROWS rows by WAVES waves; one instruction covers 8 rows.
template <int ROWS, int WAVES>
struct KcTile {
    static constexpr int kInstr = ROWS / 8 / WAVES, kBytes = ROWS * 128;
    static_assert(kInstr >= 1 && ROWS % (8 * WAVES) == 0, "every wave issues the same number of DMA instructions");
    const char* base;     // first row
    uint32_t bytes;       // of the rows that exist, from base
    uint32_t off[kInstr];
    int col;              // this lane's first contraction value within a step
    int len;              // contraction length
    __device__ __forceinline__ KcTile(const void* p, int rows, int ld, int length, int wave, int lane) {
        base = static_cast<const char*>(p);
        bytes = (uint32_t)max(min(rows, ROWS), 0) * (uint32_t)(ld * 2);
        len = bytes ? length : 0;
        const int r0 = wave * 8 + (lane >> 3), chunk = (lane & 7) ^ kc_swz(r0);
        col = chunk * 8;
#pragma unroll
        for (int j = 0; j < kInstr; ++j) {
            static_assert(kInstr == 1 || WAVES % 2 == 0, "the swizzle must not change with j");
            off[j] = (uint32_t)(r0 + j * WAVES * 8) * (uint32_t)(ld * 2) + chunk * 16;
        }
    }
    // What the DMA of step s needs: the descriptor, and whether this lane lies past the end of the rows.
    struct Step {
        u32x4 desc;
        bool cut;
    };
    __device__ __forceinline__ Step step(int s) const {
        const int k0 = s * kStepK;
        const bool live = k0 < len;
        // len is a multiple of 8: a lane's 16 bytes are all inside or all past the end
        return Step{buffer_of(base + (live ? (size_t)k0 * 2 : 0), live ? bytes - (uint32_t)k0 * 2u : 0u), k0 + col >= len};
    }
    // DMA instruction j of a step into LDS at `lds` (the operand's tile of a stage)
    __device__ __forceinline__ void load(const Step& t, int j, uint32_t lds, int wave) const {
        dma_rows(t.desc, t.cut ? kPastEnd : off[j], lds + (wave + j * WAVES) * 1024);
    }
};

// The DMA of one KS operand tile of 64 contraction rows x W columns: what depends on the lane, and what depends on
// the tile.
template <int W, int WAVES>
struct KsLanes {
    static constexpr int kRowsPerInstr = 512 / W, kInstr = kStepK / kRowsPerInstr / WAVES, kBytes = W * 128;
    static_assert(W >= 128, "eight 32-byte pairs to swizzle");
    static_assert(kInstr >= 1 && (kInstr == 1 || (kRowsPerInstr * WAVES) % 16 == 0), "the swizzle must not change with j");
    uint32_t off[kInstr];
    __device__ __forceinline__ KsLanes(int ld, int wave, int lane) {
        const int r0 = wave * kRowsPerInstr + lane / (W / 8), pos = lane % (W / 8);
        const int chunk = (((pos >> 1) ^ ks_swz(r0)) << 1) | (pos & 1);
#pragma unroll
        for (int j = 0; j < kInstr; ++j) off[j] = (uint32_t)(r0 + j * WAVES * kRowsPerInstr) * (uint32_t)(ld * 2) + chunk * 16;
    }
    __device__ __forceinline__ void load(u32x4 desc, int j, uint32_t lds, int wave) const {
        dma_rows(desc, off[j], lds + (wave + j * WAVES) * 1024);
    }
};
struct KsWhere {
    const char* base;     // contraction row 0, first column of the tile
    uint32_t ldb, skip;   // bytes of a memory row; bytes before the tile's first column
    int len;              // contraction rows, 0 for a tile behind the last column
    __device__ __forceinline__ KsWhere(const void* p, int col0, int ld, int length) {
        ldb = (uint32_t)ld * 2u;
        skip = (uint32_t)col0 * 2u;
        base = static_cast<const char*>(p) + skip;
        len = col0 < ld ? length : 0;
    }
    __device__ __forceinline__ u32x4 step(int s) const {
        const int k0 = s * kStepK, left = min(len - k0, kStepK);
        return buffer_of(base + (left > 0 ? (size_t)k0 * ldb : 0), left > 0 ? (uint32_t)left * ldb - skip : 0u);
    }
};
template <int W, int WAVES>
struct KsTile {
    using Step = u32x4;
    KsLanes<W, WAVES> lanes;
    KsWhere where;
    __device__ __forceinline__ KsTile(const void* p, int col0, int ld, int length, int wave, int lane)
        : lanes(ld, wave, lane), where(p, col0, ld, length) {}
    __device__ __forceinline__ Step step(int s) const { return where.step(s); }
    __device__ __forceinline__ void load(const Step& t, int j, uint32_t lds, int wave) const { lanes.load(t, j, lds, wave); }
};

// One operand of a product tile.  KC: `p` points at the tile's first row, `extent` rows exist from there on.  KS:
// `p` points at contraction row 0, the tile starts at column `extent`.
struct Operand {
    const uint16_t* p;
    int extent, ld, len;      // ld: values of a memory row; len: contraction length
};
// The part of an operand tile that starts at its row (column) `at`
template <bool kKs, int ROWS, int WAVES>
struct PartOf {
    using Type = KcTile<ROWS, WAVES>;
    static __device__ __forceinline__ Type make(const Operand& o, int at, int wave, int lane) {
        return Type(o.p + (size_t)at * o.ld, o.extent - at, o.ld, o.len, wave, lane);
    }
};
template <int ROWS, int WAVES>
struct PartOf<true, ROWS, WAVES> {
    using Type = KsTile<ROWS, WAVES>;
    static __device__ __forceinline__ Type make(const Operand& o, int at, int wave, int lane) {
        return Type(o.p, o.extent + at, o.ld, o.len, wave, lane);
    }
};

// Fragment (16 rows x 32 contraction values) of a KC tile: row block rb, half kk of the step.
__device__ __forceinline__ i32x4 kc_frag(const uint8_t* tile, int rb, int kk, int lane) {
    const int r = lane & 15;
    return *reinterpret_cast<const i32x4*>(tile + (rb * 16 + r) * 128 + ((((lane >> 4) + 4 * kk) ^ kc_swz(r)) << 4));
}
// Fragment of a KS tile: column block cb (16 columns), half kk.
template <int W>
__device__ __forceinline__ i32x4 ks_frag(const uint8_t* tile, int cb, int kk, int lane) {
    const int r = kk * 32 + (lane >> 4) * 8 + ((lane & 15) >> 2);
    const uint8_t* p = tile + r * (W * 2) + ((cb ^ ks_swz(r)) << 5) + (lane & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(void*)const_cast<uint8_t*>(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(void*)const_cast<uint8_t*>(p + 4 * W * 2));
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return i32x4{(int)a[0], (int)a[1], (int)b[0], (int)b[1]};
}

// ---------------------------------------------------------------- groups
// Rows of group e: clamped into 0 .. rows, a decreasing pair is empty; `bad` collects broken entries.
__device__ __forceinline__ void group_rows(const int32_t* off, int e, int rows, int& lo, int& cnt, bool& bad) {
    const int a = off[e], b = off[e + 1];
    bad |= a < 0 || b < a || b > rows;
    lo = min(max(a, 0), rows);
    cnt = max(min(max(b, 0), rows) - lo, 0);
}

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_prefix(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

struct TileAt {
    int g;       // group
    int lo;      // its first row
    int cnt;     // its rows
    int mt, nt;  // row tile and column tile within the group
};

// The groups' row tiles (BM rows each) times `ntn` column tiles, in this order: by group; within a group by
// bands of `band` column tiles; within a band row tile by row tile.  Neighbouring numbers share their row
// or their weight tiles.  All lanes take part; the result is wave-uniform.
template <int BM>
struct TileMap {
    const int32_t* off;
    int groups, rows, ntn, band;
    int first_tiles;   // per lane: row tiles of group `lane` (groups 0..63)
    int total;         // all tiles
    __device__ __forceinline__ TileMap(const int32_t* o, int g, int r, int n, int bd, int lane, uint32_t* status) {
        off = o;
        groups = g;
        rows = r;
        ntn = n;
        band = bd;
        int sum = 0;
        bool bad = false;
        first_tiles = 0;
        for (int e0 = 0; e0 < groups; e0 += 64) {
            int lo, cnt = 0;
            if (e0 + lane < groups) group_rows(off, e0 + lane, rows, lo, cnt, bad);
            const int t = (cnt + BM - 1) / BM;
            if (e0 == 0) first_tiles = t;
            sum += t;
        }
        total = __builtin_amdgcn_readfirstlane(__shfl(wave_prefix(sum, lane), 63)) * ntn;
        if (bad && status) atomicOr(status, MEGA_MOE_STATUS_BAD_LAYOUT);
    }
    __device__ __forceinline__ TileAt at(int tile, int lane) const {
        int before = 0;      // row tiles of the groups before this batch of 64
        TileAt w{-1, 0, 0, 0, 0};
        const int row_tile = tile / ntn;
        for (int e0 = 0; e0 < groups; e0 += 64) {
            int t = first_tiles;
            if (e0) {
                int lo, cnt = 0;
                bool bad = false;
                if (e0 + lane < groups) group_rows(off, e0 + lane, rows, lo, cnt, bad);
                t = (cnt + BM - 1) / BM;
            }
            const int incl = wave_prefix(t, lane) + before;
            const uint64_t hit = __ballot(incl > row_tile);
            if (hit) {
                const int l = __ffsll((unsigned long long)hit) - 1;
                const int tiles = __builtin_amdgcn_readfirstlane(__shfl(t, l));
                const int start = __builtin_amdgcn_readfirstlane(__shfl(incl, l)) - tiles;
                w.g = e0 + l;
                bool bad = false;
                group_rows(off, w.g, rows, w.lo, w.cnt, bad);
                w.lo = __builtin_amdgcn_readfirstlane(w.lo);
                w.cnt = __builtin_amdgcn_readfirstlane(w.cnt);
                const int li = tile - start * ntn, per_band = tiles * band;
                const int b = li / per_band, in = li - b * per_band;
                const int width = min(band, ntn - b * band);
                w.mt = in / width;
                w.nt = b * band + in - w.mt * width;
                return w;
            }
            before = __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
        }
        return w;
    }
};

// Work-group b of a launch goes to XCD b % 8: give every XCD one run of consecutive tiles, so that the tiles
// that share operands meet in one L2.  Returns -1 for a work-group past the tiles.
__device__ __forceinline__ int xcd_tile(int block, int total) {
    const int per = (total + 7) >> 3, i = block >> 3, t = (block & 7) * per + i;
    return i < per && t < total ? t : -1;
}

}  // namespace mm
