// Pieces shared by the operators that work on rows (norm.hip, activation.hip), gfx950 only: eight columns of a row as
// a lane's unit, reductions over the 16 lanes of a 128-column block, and the 8-bit form.
//
// A lane moves 8 values at a time (16 bytes of a 16-bit type), so 16 lanes, which DPP reduces without LDS, hold the 128
// columns of one scale.  Rows of any length and any alignment of the element type are taken: the hardware loads and
// stores 16 bytes at any address, and only the last, partial unit of a row goes value by value.
//
// The 8-bit form: e4m3 codes and, for each 128 columns, the scale 2^ceil(log2(largest / 448)), which is the smallest
// power of two that saturates no value.  A power of two costs no accuracy (the codes keep four significant bits whatever
// the scale; a finer scale would only move the end of their range), and code * scale is exact in bf16 and in fp16, so
// that restored values can enter matrix products without a second rounding.  A block that holds an infinity or a NaN
// becomes NaN throughout: the codes have no infinity, and an overflow must not look like a number.
#pragma once

#include "gemm_tiles.h"

namespace mm {

struct Fp32 {
    static constexpr bool kNarrow = false;
};

typedef u32x4 u32x4_any __attribute__((aligned(2)));      // 16 bytes at an address of 2-byte alignment
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// Loads and stores that leave the caches to others (non-temporal) or not.  Rows are written past the caches everywhere:
// 32768 rows of 2048 columns in SwiGLU 76 -> 58 us, of 7168 columns in the norm 372 -> 353, restored 133 -> 105, and what reads
// them next takes no longer (SwiGLU and the product behind it 302 -> 296 us at 8192 rows, 850 and 854 at 32768).
template <bool kOnce, class V>
__device__ __forceinline__ V read(const V* p) {
    if constexpr (kOnce) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool kOnce, class V, class W>
__device__ __forceinline__ void write(V* p, W v) {
    if constexpr (kOnce) __builtin_nontemporal_store((V)v, p);
    else *p = v;
}

// Eight values as they are in memory, and the way to them: load n >= 8 at once, or the n < 8 that exist with zeros
// behind them (n <= 0 reads nothing).  opaque(): what was computed from them before is not known to the compiler any more.
template <class T>
struct Row8 {
    static constexpr int kBytes = 2;
    u32x4 w;
    template <bool kOnce = false>
    static __device__ __forceinline__ Row8 load(const void* base, size_t at, int n) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        Row8 r;
        if (n >= 8) {
            r.w = read<kOnce>(reinterpret_cast<const u32x4_any*>(p));
        } else {
            r.w = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) r.w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        }
        return r;
    }
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = T::low(w[i]);
            v[2 * i + 1] = T::high(w[i]);
        }
    }
    static __device__ __forceinline__ void store(void* base, size_t at, int n, const float (&v)[8]) {
        uint16_t* p = static_cast<uint16_t*>(base) + at;
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = T::pack(v[2 * i], v[2 * i + 1]);
        if (n >= 8) {
            write<true>(reinterpret_cast<u32x4_any*>(p), r);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) p[i] = (uint16_t)(r[i / 2] >> (16 * (i & 1)));
        }
    }
};
template <>
struct Row8<Fp32> {
    static constexpr int kBytes = 4;
    u32x4 a, b;
    template <bool kOnce = false>
    static __device__ __forceinline__ Row8 load(const void* base, size_t at, int n) {
        const uint32_t* p = static_cast<const uint32_t*>(base) + at;
        Row8 r;
        if (n >= 8) {
            r.a = read<kOnce>(reinterpret_cast<const u32x4_any4*>(p));
            r.b = read<kOnce>(reinterpret_cast<const u32x4_any4*>(p + 4));
        } else {
            r.a = r.b = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) (i < 4 ? r.a : r.b)[i & 3] = p[i];
        }
        return r;
    }
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(a), "+v"(b)); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(a[i]);
            v[4 + i] = __uint_as_float(b[i]);
        }
    }
    static __device__ __forceinline__ void store(void* base, size_t at, int n, const float (&v)[8]) {
        uint32_t* p = static_cast<uint32_t*>(base) + at;
        if (n >= 8) {
            u32x4 lo, hi;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = __float_as_uint(v[i]);
                hi[i] = __float_as_uint(v[4 + i]);
            }
            write<true>(reinterpret_cast<u32x4_any4*>(p), lo);
            write<true>(reinterpret_cast<u32x4_any4*>(p + 4), hi);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) p[i] = __float_as_uint(v[i]);
        }
    }
};

// Eight codes; get() multiplies by their scale.
struct Codes8 {
    u32x2 w;
    template <bool kOnce>
    static __device__ __forceinline__ Codes8 load(const void* base, size_t at, int n) {
        const uint8_t* p = static_cast<const uint8_t*>(base) + at;
        Codes8 r;
        if (n >= 8) {
            r.w = read<kOnce>(reinterpret_cast<const u32x2_any*>(p));
        } else {
            r.w = u32x2{0, 0};
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) r.w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
        }
        return r;
    }
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ void get(float scale, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            v[4 * i] = lo[0] * scale;
            v[4 * i + 1] = lo[1] * scale;
            v[4 * i + 2] = hi[0] * scale;
            v[4 * i + 3] = hi[1] * scale;
        }
    }
    // v / scale in codes, inverse = 1 / scale (exact, a power of two): at most 448 in magnitude, or NaN
    template <bool kOnce>
    static __device__ __forceinline__ void store(void* base, size_t at, int n, const float (&v)[8], float inverse) {
        uint8_t* p = static_cast<uint8_t*>(base) + at;
        u32x2 r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inverse, v[4 * i + 1] * inverse, 0, false);
            r[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inverse, v[4 * i + 3] * inverse, lo, true);
        }
        if (n >= 8) {
            write<kOnce>(reinterpret_cast<u32x2_any*>(p), r);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) p[i] = (uint8_t)(r[i / 4] >> (8 * (i & 3)));
        }
    }
};

// ---------------------------------------------------------------- reductions over 16 lanes (a DPP row)
template <int kBy>
__device__ __forceinline__ uint32_t turned(uint32_t v) {      // the value of the lane kBy before, around the 16
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + kBy, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, turned<8>(v));
    v = max(v, turned<4>(v));
    v = max(v, turned<2>(v));
    return max(v, turned<1>(v));
}
template <int kBy>
__device__ __forceinline__ double turned(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, u32x2{turned<kBy>(w[0]), turned<kBy>(w[1])});
}
// The same bits in all lanes: after each step the values repeat with half the period, and additions commute.
__device__ __forceinline__ double sum16(double v) {
    v += turned<8>(v);
    v += turned<4>(v);
    v += turned<2>(v);
    return v + turned<1>(v);
}
__device__ __forceinline__ double sum64(double v) {
    v = sum16(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Bits of the largest magnitude: NaN above infinity above numbers.
__device__ __forceinline__ uint32_t largest(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}
// The scale of a block from its largest magnitude's bits, and its inverse (NaN where the block holds no finite number
// throughout, with a scale of 1).  448 = 1.75 * 2^8, so the exponent is 8 below the largest one's, or 7 where its mantissa
// is over 1.75; 2^-126 at least, so that scale and inverse are ordinary numbers.
struct Scale {
    float scale, inverse;
    bool end;       // the largest one would round to 2^128
    __device__ __forceinline__ explicit Scale(uint32_t top) {
        end = top >= 0x7F780000u;
        const int e = max((int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 1);
        const bool finite = top < 0x7F800000u;
        scale = finite ? __uint_as_float((uint32_t)e << 23) : 1.0f;
        inverse = __uint_as_float(finite ? (uint32_t)(254 - e) << 23 : 0x7FC00000u);
    }
    // codes of eight values; at the very end of fp32's range the largest four-bit number below 2^128 stands for what is above it
    template <bool kOnce>
    __device__ __forceinline__ void store(void* codes, size_t at, int n, float (&v)[8]) const {
        if (end) {
            const float most = __uint_as_float(0x7F700000u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] > most ? most : v[i] < -most ? -most : v[i];
        }
        Codes8::store<kOnce>(codes, at, n, v, inverse);
    }
};

// Whether a pass reads more than three quarters of the last-level cache (256 MB), which its outputs share: most of what it
// reads is then in no cache, and is read past them.  Measured past them and not: 32768 rows, quantize of 7168 columns 119 and 132 us,
// the norm's gradient 354 and 362, SwiGLU of 2048 with its input kept 85 and 100; 16384 rows of 7168 columns (235 MB), quantize, 61
// and 67, 12288 rows 47 and 45; 4096 rows 17.6 and 15.7, the norm's gradient 48 and 42, SwiGLU 14 and 12.
inline bool beyond_cache(uint64_t bytes) { return bytes > (uint64_t)192 << 20; }

constexpr int kScaleCols = 128;      // columns of one scale
__host__ __device__ inline int scale_blocks(int cols) { return (cols + kScaleCols - 1) / kScaleCols; }

}  // namespace mm
