// Products grouped by expert with ragged rows, and their gradients (include/mega_moe_ops.h):
//   forward          y[m]  = x[m] w[e]^T      P = x rows (KC),  Q = w rows (KC),   contraction k
//   backward_rows    dx[m] = dy[m] w[e]       P = dy rows (KC), Q = w columns (KS), contraction n
//   backward_weight  dw[e] = dy_e^T x_e       P = dy columns (KS), Q = x columns (KS), contraction rows
// The row-major weights are read as they are in all three: where the contraction runs down the memory rows
// the fragments are transposed on their way out of LDS.
//
// Measured, bf16.  Many rows (32768 x 4096 x 7168 over 32 groups): 1.69 ms, 1140 TFLOP/s.  The loop itself reaches 1430
// where one group fills its tiles (8192 rows, 335 us); the rest goes to the groups' last tiles, to the ninth and tenth
// round of tiles on 256 CUs, and to the clock, which the DMA's power takes from 2.17 to 1.89 GHz.  Few rows stream the
// weights: 1024 x 7168 x 2048 over 32 groups 171 us (5.6 TB/s), eight rows for eight groups of 4096 x 7168 78 us (6.0).
// The gradient of rows (8192 rows, 32 x 4096 x 1536: 148 us, 700 TFLOP/s, 3.3 TB/s) has the forward's bounds, and both
// at once.  The gradient of weights of short groups writes as much as it multiplies, and the two share the CUs' time:
// 16384 rows, 32 x 4096 x 7168, fp32, 1.38 ms for 962 GFLOP and 4.1 GB.
#include <type_traits>

#include "codes_loop.h"
#include "gemm_kernels.h"

namespace mm {
namespace {

struct GroupedArgs {
    const uint16_t* p;     // x or dy
    const uint16_t* q;     // w, or x (backward_weight)
    void* out;
    const int32_t* off;
    uint32_t* status;
    int rows, n, k, groups;
    int accumulate;
    int parts;             // backward_weight: parts of a group's rows, each with its own output
};

// One tile of out = P Q^T with loop L; `out` points at the tile's first row and column, rows and cols exist there.
template <class L, class T>
__device__ __forceinline__ void rows_tile(const Operand& P, const Operand& Q, uint16_t* out, int rows, int cols, int ld,
                                          uint8_t* smem, int wave, int lane) {
    typename L::Acc acc[L::QI][L::MI];
    L::run(P, Q, smem, wave, lane, acc);
    store_halves<L, T>(acc, out, rows, cols, ld, smem, wave, lane);
}

// forward / backward_rows: one BM x BN tile of a group's rows per work-group.  H is a loop over half as many rows,
// for the last tile of a group where it has no more: groups end anywhere, and a whole tile for their last rows
// costs half a tile per group on average.
template <class L, class H, class T, bool kBackward, int BM, int BN>
__global__ __launch_bounds__(L::kThreads) void grouped_rows_kernel(GroupedArgs a) {
    static_assert(H::kThreads == L::kThreads, "one launch");
    __shared__ __align__(1024) uint8_t smem[L::kLds > H::kLds ? L::kLds : H::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cols = kBackward ? a.k : a.n, depth = kBackward ? a.n : a.k;
    const TileMap<BM> map(a.off, a.groups, a.rows, (cols + BN - 1) / BN, 8, lane, blockIdx.x ? nullptr : a.status);
    const int tile = xcd_tile(blockIdx.x, map.total);
    if (tile < 0) return;
    const TileAt w = map.at(tile, lane);
    if (w.g < 0) return;
    const int m0 = w.mt * BM, q0 = w.nt * BN, rows = w.cnt - m0;
    const uint16_t* wg = a.q + (size_t)w.g * a.n * a.k;
    const Operand P{a.p + (size_t)(w.lo + m0) * depth, rows, depth, depth};
    const Operand Q = kBackward ? Operand{wg, q0, a.k, a.n} : Operand{wg + (size_t)q0 * a.k, a.n - q0, a.k, a.k};
    uint16_t* out = static_cast<uint16_t*>(a.out) + (size_t)(w.lo + m0) * cols + q0;
    if (!std::is_same<L, H>::value && rows <= BM / 2)
        rows_tile<H, T>(P, Q, out, rows, cols - q0, cols, smem, wave, lane);
    else
        rows_tile<L, T>(P, Q, out, rows, cols - q0, cols, smem, wave, lane);
}

// The nth longest of at most 64 groups (equal lengths: the lower one first).
__device__ __forceinline__ int group_by_length(const int32_t* off, int groups, int rows, int nth, int lane) {
    int lo, cnt = -1;
    bool bad = false;
    if (lane < groups) group_rows(off, lane, rows, lo, cnt, bad);
    int before = 0;
    for (int e = 0; e < groups; ++e) {
        const int c = __builtin_amdgcn_readlane(cnt, e);
        before += c > cnt || (c == cnt && e < lane);
    }
    return __ffsll((unsigned long long)__ballot(lane < groups && before == nth)) - 1;
}

// backward_weight: one BM x BN tile of dw[e] per work-group
template <class L, class T, bool kFp32, int BM, int BN>
__global__ __launch_bounds__(L::kThreads) void grouped_weight_kernel(GroupedArgs a) {
    __shared__ __align__(1024) uint8_t smem[L::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ntm = (a.n + BM - 1) / BM, ntq = (a.k + BN - 1) / BN;
    // work-groups b with equal b % 8 share an XCD: each XCD takes an eighth of every group's tiles, since the
    // groups differ in length (whole groups per XCD left the XCDs of short groups idle half of the time)
    const int per = (ntm * ntq + 7) >> 3, part = (int)((blockIdx.x >> 3) % a.parts), b = (int)((blockIdx.x >> 3) / a.parts), nth = b / per,
              li = (blockIdx.x & 7) * per + b - nth * per;
    if (nth >= a.groups || li >= ntm * ntq) return;
    const int g = a.groups <= 64 ? group_by_length(a.off, a.groups, a.rows, nth, lane) : nth;
    // bands of 8 row tiles, as the row products have bands of column tiles
    const int band = li / (8 * ntq), in = li - band * 8 * ntq, width = min(8, ntm - band * 8);
    const int qt = in / width, m0 = (band * 8 + in - qt * width) * BM, q0 = qt * BN;
    int lo, cnt;
    bool bad = false;
    group_rows(a.off, g, a.rows, lo, cnt, bad);
    lo = __builtin_amdgcn_readfirstlane(lo);
    cnt = __builtin_amdgcn_readfirstlane(cnt);
    if (bad && li == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, MEGA_MOE_STATUS_BAD_LAYOUT);
    if (cnt == 0 && a.accumulate && a.parts == 1) return;
    if (a.parts > 1) {
        const int share = ((cnt + kStepK - 1) / kStepK + a.parts - 1) / a.parts * kStepK, from = min(part * share, cnt);
        lo += from;
        cnt = min(cnt - from, share);
    }
    typename L::Acc acc[L::QI][L::MI];
    const Operand P{a.p + (size_t)lo * a.n, m0, a.n, cnt}, Q{a.q + (size_t)lo * a.k, q0, a.k, cnt};
    L::run(P, Q, smem, wave, lane, acc);
    const size_t at = (((size_t)part * a.groups + g) * a.n + m0) * a.k + q0;
    if constexpr (kFp32) {
        float* out = static_cast<float*>(a.out) + at;
        store_tile<L, 4>(
            acc, smem, a.n - m0, a.k - q0, wave, lane, [](uint8_t* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; },
            [&](int m, int c, i32x4 v) {
                f32x4* o = reinterpret_cast<f32x4*>(out + (size_t)m * a.k + c);
                f32x4 sum = __builtin_bit_cast(f32x4, v);
                if (a.accumulate) sum += *o;
                *o = sum;
            });
    } else {
        store_halves<L, T>(acc, static_cast<uint16_t*>(a.out) + at, a.n - m0, a.k - q0, a.k, smem, wave, lane);
    }
}

// backward_weight with enough large tiles for every CU: a stream of them per work-group, 32 work-groups to an XCD.
// Each XCD takes an eighth of every group's tiles, longest group first, and its work-groups take turns.
constexpr int kStreams = 32;
template <class T, bool kFp32, bool kLines>
__global__ __launch_bounds__(512) void grouped_weight_stream_kernel(GroupedArgs a) {
    constexpr int kBytes = kFp32 ? 4 : 2;
    using S = KsStream<T, kBytes, kLines>;
    static_assert(S::kThreads == 512, "one launch");
    __shared__ __align__(1024) uint8_t smem[S::kLds];
    // the groups in the order of their tiles: longest first where 64 lanes can rank them (long and short ones in turn,
    // so that stores meet MFMAs, took longer: 1.49 ms against 1.43 with skewed groups)
    __shared__ int order_g[MEGA_MOE_MAX_LOCAL_EXPERTS], order_first[MEGA_MOE_MAX_LOCAL_EXPERTS],
        order_rows[MEGA_MOE_MAX_LOCAL_EXPERTS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ntm = (a.n + S::BM - 1) / S::BM, ntq = (a.k + S::BN - 1) / S::BN, per = (ntm * ntq + 7) >> 3;
    bool bad = false;
    for (int e = threadIdx.x; e < a.groups; e += S::kThreads) {
        int lo, cnt, place = e;
        group_rows(a.off, e, a.rows, lo, cnt, bad);
        if (a.groups <= 64) {
            place = 0;
            for (int o = 0; o < a.groups; ++o) {
                const int c = __builtin_amdgcn_readlane(cnt, o);
                place += c > cnt || (c == cnt && o < e);
            }
        }
        order_g[place] = e;
        order_first[place] = lo;
        order_rows[place] = cnt;
    }
    if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, MEGA_MOE_STATUS_BAD_LAYOUT);
    __syncthreads();
    const int xcd = blockIdx.x & 7, total = a.groups * per;
    int at = blockIdx.x >> 3;
    const auto next = [&]() __attribute__((always_inline)) {
        int nth = 0, li = 0, rows = 0;
        bool found = false;
        while (!found && at < total) {
            nth = __builtin_amdgcn_readfirstlane(at / per);
            li = __builtin_amdgcn_readfirstlane(xcd * per + at - nth * per);
            at = __builtin_amdgcn_readfirstlane(at + kStreams);
            rows = __builtin_amdgcn_readfirstlane(order_rows[nth]);
            found = __builtin_amdgcn_readfirstlane(li < ntm * ntq && (rows > 0 || !a.accumulate));
        }
        const int g = __builtin_amdgcn_readfirstlane(order_g[nth]), first = __builtin_amdgcn_readfirstlane(order_first[nth]);
        const int band = li / (8 * ntq), in = li - band * 8 * ntq, width = min(8, ntm - band * 8);
        const int qt = in / width, m0 = (band * 8 + in - qt * width) * S::BM, q0 = qt * S::BN;
        return S::of(found, a.p + (size_t)first * a.n, m0, a.q + (size_t)first * a.k, q0, rows,
                     static_cast<char*>(a.out) + (((size_t)g * a.n + m0) * a.k + q0) * kBytes, a.n - m0, a.k - q0);
    };
    S::run(next, a.n, a.k, a.k, smem, wave, lane, [&](const char* p, bool exists, i32x4 v) {
        if constexpr (kFp32)
            if (a.accumulate && exists)
                v = __builtin_bit_cast(i32x4, __builtin_bit_cast(f32x4, v) + *reinterpret_cast<const f32x4*>(p));
        return v;
    });
}

// backward_weight from 8-bit rows: one 256 x 128 tile of dw[e] per work-group, tiles to XCDs as above.  The launch is no
// stream of tiles: a work-group that ends leaves its stores on their way and its place on the CU to the next one.
struct CodesArgs {
    GroupedArgs g;               // p: dy
    const uint8_t* codes;
    const float* scales;
};
template <class T, bool kFp32>
__global__ __launch_bounds__(256, 2) void grouped_codes_kernel(CodesArgs c) {
    using L = CodesLoop<T>;
    const GroupedArgs& a = c.g;
    __shared__ __align__(1024) uint8_t smem[L::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ntm = (a.n + L::BM - 1) / L::BM, ntq = (a.k + L::BN - 1) / L::BN;
    const int per = (ntm * ntq + 7) >> 3, part = (int)((blockIdx.x >> 3) % a.parts), b = (int)((blockIdx.x >> 3) / a.parts), nth = b / per,
              li = (blockIdx.x & 7) * per + b - nth * per;
    if (nth >= a.groups || li >= ntm * ntq) return;
    const int g = a.groups <= 64 ? group_by_length(a.off, a.groups, a.rows, nth, lane) : nth;
    const int band = li / (4 * ntq), in = li - band * 4 * ntq, width = min(4, ntm - band * 4);
    const int qt = in / width, m0 = (band * 4 + in - qt * width) * L::BM, q0 = qt * L::BN;
    int lo, cnt;
    bool bad = false;
    group_rows(a.off, g, a.rows, lo, cnt, bad);
    lo = __builtin_amdgcn_readfirstlane(lo);
    cnt = __builtin_amdgcn_readfirstlane(cnt);
    if (bad && li == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, MEGA_MOE_STATUS_BAD_LAYOUT);
    if (cnt == 0 && a.accumulate && a.parts == 1) return;
    if (a.parts > 1) {
        const int share = ((cnt + L::kDepth - 1) / L::kDepth + a.parts - 1) / a.parts * L::kDepth, from = min(part * share, cnt);
        lo += from;
        cnt = min(cnt - from, share);
    }
    const int blocks = (a.k + 127) / 128;
    typename L::Acc acc[L::QI][L::MI];
    const uint16_t* p = a.p + (size_t)lo * a.n;
    const uint8_t* x = c.codes + (size_t)lo * a.k;
    const float* scales = c.scales + (size_t)lo * blocks;
    L::run(p, a.n, m0, x, a.k, q0, scales, blocks, cnt, smem, wave, lane, acc);
    const size_t at = (((size_t)part * a.groups + g) * a.n + m0) * a.k + q0;
    if constexpr (kFp32) {
        float* out = static_cast<float*>(a.out) + at;
        store_tile<L, 4>(
            acc, smem, a.n - m0, a.k - q0, wave, lane, [](uint8_t* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; },
            [&](int m, int col, i32x4 v) {
                f32x4* o = reinterpret_cast<f32x4*>(out + (size_t)m * a.k + col);
                f32x4 sum = __builtin_bit_cast(f32x4, v);
                if (a.accumulate) sum += *o;
                *o = sum;
            });
    } else {
        store_halves<L, T>(acc, static_cast<uint16_t*>(a.out) + at, a.n - m0, a.k - q0, a.k, smem, wave, lane);
    }
}

// dw = the parts added up in their order (dw += with accumulate); values is a multiple of 8
template <class T, bool kFp32>
__global__ __launch_bounds__(256) void grouped_join_kernel(const float* parts, int n_parts, size_t values, void* out,
                                                           int accumulate) {
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < values; i += (size_t)gridDim.x * 1024) {
        f32x4 v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int s = 0; s < n_parts; ++s) v += *reinterpret_cast<const f32x4*>(parts + s * values + i);
        if constexpr (kFp32) {
            f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + i);
            *o = accumulate ? *o + v : v;
        } else {
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) = u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
        }
    }
}

bool aligned16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }

bool sizes_supported(int64_t rows, int32_t n, int32_t k, int32_t groups) {
    return rows <= MEGA_MOE_MAX_GROUP_ROWS && n >= 8 && n <= MEGA_MOE_MAX_GROUP_COLS && n % 8 == 0 && k >= 8 &&
           k <= MEGA_MOE_MAX_GROUP_COLS && k % 8 == 0 && groups >= 1 && groups <= MEGA_MOE_MAX_LOCAL_EXPERTS;
}

int32_t check_grouped(const void* p, const void* q, const int32_t* off, const void* out, int64_t rows, int32_t n,
                      int32_t k, int32_t groups, int32_t dtype, const uint32_t* status, bool weight) {
    if (rows < 0 || n < 0 || k < 0 || groups < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!sizes_supported(rows, n, k, groups) || (dtype != MEGA_MOE_BF16 && dtype != MEGA_MOE_FP16))
        return MEGA_MOE_ERR_UNSUPPORTED;
    if (!off || ((uintptr_t)off & 3u) || ((uintptr_t)status & 3u)) return MEGA_MOE_ERR_INVALID_ARG;
    const bool any = rows > 0;
    if ((any && !aligned16(p)) || ((any || !weight) && !aligned16(q)) || ((any || weight) && !aligned16(out)))
        return MEGA_MOE_ERR_INVALID_ARG;
    return MEGA_MOE_OK;
}

template <class L, class H, class T, bool kBackward, int BM, int BN>
hipError_t launch_rows_with(const GroupedArgs& a, hipStream_t st) {
    const int64_t tiles = ((int64_t)a.rows / BM + min(a.groups, a.rows)) * (((kBackward ? a.k : a.n) + BN - 1) / BN);
    if ((tiles + 7) * L::kThreads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((grouped_rows_kernel<L, H, T, kBackward, BM, BN>), dim3((uint32_t)((tiles + 7) / 8 * 8)),
                       dim3(L::kThreads), 0, st, a);
    return hipGetLastError();
}

template <class T, bool B>
hipError_t launch_rows(const GroupedArgs& a, hipStream_t st) {
    using Wide = TileLoop<T, false, B, 128, 256, 2, 4, 3>;
    using Low = TileLoop<T, false, B, 64, 256, 1, 8, 3>;
    using Square = TileLoop<T, false, B, 128, 128, 2, 4, 4>;
    using Mid = TileLoop<T, false, B, 64, 128, 1, 4, 3>;
    using Small = TileLoop<T, false, B, 32, 128, 1, 4, 4>;
    // a KS operand needs 128 columns: the narrower shapes are the forward's only
    const int shape = pick_row_shape(a.rows, B ? a.k : a.n, B ? a.n : a.k, a.groups, B ? kShapeHalved + 1 : kShapeDeep + 1);
    if (shape == kShape256)
        return launch_rows_with<QuadLoop<T, false, B, 256, 256, 4, 2>, Wide, T, B, 256, 256>(a, st);
    if (shape == kShape128) return launch_rows_with<Wide, Low, T, B, 128, 256>(a, st);
    if (shape == kShapeSquare)
        return launch_rows_with<Square, TileLoop<T, false, B, 64, 128, 2, 4, 6>, T, B, 128, 128>(a, st);
    if (shape == kShape64) return launch_rows_with<Mid, Mid, T, B, 64, 128>(a, st);
    if (shape == kShape32) return launch_rows_with<Small, Small, T, B, 32, 128>(a, st);
    using Halved = TileLoop<T, false, B, 64, 128, 1, 4, 3, 2>;
    if (shape == kShapeHalved) return launch_rows_with<Halved, Halved, T, B, 64, 128>(a, st);
    if constexpr (!B) {
        using Least = TileLoop<T, false, false, 32, 64, 1, 4, 5>;
        using Deep = TileLoop<T, false, false, 32, 64, 1, 4, 3, 4>;
        if (shape == kShapeLeast) return launch_rows_with<Least, Least, T, false, 32, 64>(a, st);
        return launch_rows_with<Deep, Deep, T, false, 32, 64>(a, st);
    }
    return hipErrorInvalidValue;
}

template <class L, class T, bool kFp32, int BM, int BN>
hipError_t launch_weight_with(const GroupedArgs& a, hipStream_t st) {
    const int64_t tiles = (int64_t)((a.n + BM - 1) / BM) * ((a.k + BN - 1) / BN);
    hipLaunchKernelGGL((grouped_weight_kernel<L, T, kFp32, BM, BN>),
                       dim3((uint32_t)((tiles + 7) / 8 * 8 * a.groups * a.parts)), dim3(L::kThreads), 0, st, a);
    return hipGetLastError();
}

// 256 x 256 tiles where they fill the CUs (16384 rows, 32 x 4096 x 7168, fp32: 1.38 ms as streams of tiles, 1.44 with a
// work-group for each, 1.75 with 128 x 128).  Below that the smaller ones, four times as many, and where these leave CUs without work and the
// groups are long, the rows are split into parts of at least four steps (of an average group) that a second launch adds up.
constexpr int kWeightLarge = 192;
int64_t weight_tiles(int n, int k, int groups, int edge) {
    return (int64_t)groups * ((n + edge - 1) / edge) * ((k + edge - 1) / edge);
}
int weight_parts(int64_t rows, int n, int k, int groups) {
    if (weight_tiles(n, k, groups, 256) >= kWeightLarge) return 1;
    const int64_t by_tiles = 256 / weight_tiles(n, k, groups, 128), by_rows = rows / groups / (4 * kStepK);
    const int64_t parts = by_tiles < by_rows ? by_tiles : by_rows;
    return (int)(parts < 1 ? 1 : parts);
}

// 128 x 128 tiles: with no more than one to a CU four stages, since nothing else hides a load (1400 rows, 1768 x 592:
// 16 us against 21); with more of them two, so that two tiles share a CU (2000 rows, 4 x 1000 x 2056: 26 us against 28).
template <class T, bool kFp32>
hipError_t launch_small_weight(const GroupedArgs& a, hipStream_t st) {
    if (weight_tiles(a.n, a.k, a.groups, 128) * a.parts <= 256)
        return launch_weight_with<TileLoop<T, true, true, 128, 128, 2, 4, 4>, T, kFp32, 128, 128>(a, st);
    return launch_weight_with<TileLoop<T, true, true, 128, 128, 2, 2, 2>, T, kFp32, 128, 128>(a, st);
}

template <class T, bool kFp32>
hipError_t launch_weight(GroupedArgs a, void* workspace, hipStream_t st) {
    if (weight_tiles(a.n, a.k, a.groups, 256) >= kWeightLarge) {
        if ((uint32_t)a.k * (kFp32 ? 4u : 2u) % 128 == 0 && ((uintptr_t)a.out & 127u) == 0)
            hipLaunchKernelGGL((grouped_weight_stream_kernel<T, kFp32, true>), dim3(8 * kStreams), dim3(512), 0, st, a);
        else
            hipLaunchKernelGGL((grouped_weight_stream_kernel<T, kFp32, false>), dim3(8 * kStreams), dim3(512), 0, st, a);
        return hipGetLastError();
    }
    if (a.parts == 1) return launch_small_weight<T, kFp32>(a, st);
    void* dw = a.out;
    const int accumulate = a.accumulate;
    a.out = workspace;
    a.accumulate = 0;
    const hipError_t e = launch_small_weight<T, true>(a, st);
    if (e != hipSuccess) return e;
    const size_t values = (size_t)a.groups * a.n * a.k;
    const size_t blocks = (values + 1023) / 1024;
    hipLaunchKernelGGL((grouped_join_kernel<T, kFp32>), dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st,
                       static_cast<const float*>(workspace), a.parts, values, dw, accumulate);
    return hipGetLastError();
}

// From 8-bit rows.  Where the output has many 256 x 256 tiles for every CU, the rows are restored first and take the 16-bit
// product, whose large tiles need fewer loads for each MFMA; below that the codes are read by the product itself, and no
// 16-bit copy is made.  Restored and read as codes, bf16: 32 groups of 1024 rows, 4096 x 7168, 1881 and 1920 us; 32 of 128,
// 7168 x 2048, 225 and 301; 32 of 1024, 4096 x 1536, 428 and 412; 8 of 1024, 2048 x 2048, 79 and 68; 10 of 200, 1000 x 2056, 32 and
// 23; one of 4096, 1024 x 2048, 34 and 33.  (Rows shorter than the loads of 16 codes are restored too.)
constexpr int kCodesLarge = 2048;
bool codes_restored(int n, int k, int groups) { return k < 16 || weight_tiles(n, k, groups, 256) >= kCodesLarge; }
// 256 x 128 tiles, two to a CU; where these leave CUs without work and the groups are long, the rows are split into parts of
// at least 512 (of an average group), as many as give every CU one tile: what the second launch adds up grows with them (4096
// rows, 1024 x 2048: 33 us with one tile to a CU, 41 with two, 45 with half of one).
int64_t codes_tiles(int n, int k, int groups) { return (int64_t)groups * ((n + 255) / 256) * ((k + 127) / 128); }
int codes_parts(int64_t rows, int n, int k, int groups) {
    const int64_t by_tiles = 256 / codes_tiles(n, k, groups), by_rows = rows / groups / 512;
    const int64_t parts = by_tiles < by_rows ? by_tiles : by_rows;
    return (int)(parts < 1 ? 1 : parts);
}

template <class T, bool kFp32>
hipError_t launch_codes_tiles(const CodesArgs& a, hipStream_t st) {
    const int64_t tiles = codes_tiles(a.g.n, a.g.k, 1);
    hipLaunchKernelGGL((grouped_codes_kernel<T, kFp32>), dim3((uint32_t)((tiles + 7) / 8 * 8 * a.g.groups * a.g.parts)), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <class T, bool kFp32>
hipError_t launch_codes(CodesArgs a, void* workspace, hipStream_t st) {
    if (a.g.parts == 1) return launch_codes_tiles<T, kFp32>(a, st);
    void* dw = a.g.out;
    const int accumulate = a.g.accumulate;
    a.g.out = workspace;
    a.g.accumulate = 0;
    const hipError_t e = launch_codes_tiles<T, true>(a, st);
    if (e != hipSuccess) return e;
    const size_t values = (size_t)a.g.groups * a.g.n * a.g.k;
    const size_t blocks = (values + 1023) / 1024;
    hipLaunchKernelGGL((grouped_join_kernel<T, kFp32>), dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st,
                       static_cast<const float*>(workspace), a.g.parts, values, dw, accumulate);
    return hipGetLastError();
}

// a launch has fewer than 2^32 threads: at most 2^22 tiles of any shape
bool too_many_tiles(int64_t rows, int cols, int groups) {
    return (rows / 128 + groups) * ((cols + 127) / 128) > (int64_t)1 << 22;
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int32_t mega_moe_grouped_forward(const void* x, const void* w, const int32_t* offsets, void* y, int64_t rows, int32_t n,
                                 int32_t k, int32_t groups, int32_t dtype, uint32_t* device_status, void* stream) {
    const int32_t rc = check_grouped(x, w, offsets, y, rows, n, k, groups, dtype, device_status, false);
    if (rc) return rc;
    if (too_many_tiles(rows, n, groups)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MEGA_MOE_OK;
    const GroupedArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), y, offsets, device_status,
                        (int)rows, n, k, groups, 0, 1};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == MEGA_MOE_BF16 ? launch_rows<Bf16, false>(a, st) : launch_rows<Fp16, false>(a, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_grouped_backward_rows(const void* dy, const void* w, const int32_t* offsets, void* dx, int64_t rows,
                                       int32_t n, int32_t k, int32_t groups, int32_t dtype, uint32_t* device_status,
                                       void* stream) {
    const int32_t rc = check_grouped(dy, w, offsets, dx, rows, n, k, groups, dtype, device_status, false);
    if (rc) return rc;
    if (too_many_tiles(rows, k, groups)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MEGA_MOE_OK;
    const GroupedArgs a{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(w), dx, offsets, device_status,
                        (int)rows, n, k, groups, 0, 1};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == MEGA_MOE_BF16 ? launch_rows<Bf16, true>(a, st) : launch_rows<Fp16, true>(a, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_grouped_weight_workspace_bytes(int64_t rows, int32_t n, int32_t k, int32_t groups, uint64_t* bytes_out) {
    if (!bytes_out || rows < 0 || n < 0 || k < 0 || groups < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!sizes_supported(rows, n, k, groups)) return MEGA_MOE_ERR_UNSUPPORTED;
    const int parts = weight_parts(rows, n, k, groups);
    *bytes_out = parts > 1 ? (uint64_t)parts * groups * n * k * 4 : 0;
    return MEGA_MOE_OK;
}

int32_t mega_moe_grouped_backward_weight(const void* dy, const void* x, const int32_t* offsets, void* dw, int64_t rows,
                                         int32_t n, int32_t k, int32_t groups, int32_t dtype, int32_t out_dtype,
                                         int32_t accumulate, void* workspace, uint64_t workspace_bytes,
                                         uint32_t* device_status, void* stream) {
    const int32_t rc = check_grouped(dy, x, offsets, dw, rows, n, k, groups, dtype, device_status, true);
    if (rc) return rc;
    if (out_dtype != dtype && out_dtype != MEGA_MOE_FP32) return MEGA_MOE_ERR_UNSUPPORTED;
    if (accumulate && out_dtype != MEGA_MOE_FP32) return MEGA_MOE_ERR_UNSUPPORTED;
    // a launch has fewer than 2^32 threads
    if (weight_tiles(n, k, groups, 256) > (int64_t)1 << 21) return MEGA_MOE_ERR_UNSUPPORTED;
    const int parts = weight_parts(rows, n, k, groups);
    if (parts > 1) {
        if (!aligned16(workspace)) return MEGA_MOE_ERR_INVALID_ARG;
        if (workspace_bytes < (uint64_t)parts * groups * n * k * 4) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    const GroupedArgs a{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(x), dw, offsets, device_status,
                        (int)rows, n, k, groups, accumulate != 0, parts};
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (out_dtype == MEGA_MOE_FP32)
        e = dtype == MEGA_MOE_BF16 ? launch_weight<Bf16, true>(a, workspace, st) : launch_weight<Fp16, true>(a, workspace, st);
    else
        e = dtype == MEGA_MOE_BF16 ? launch_weight<Bf16, false>(a, workspace, st) : launch_weight<Fp16, false>(a, workspace, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_grouped_codes_workspace_bytes(int64_t rows, int32_t n, int32_t k, int32_t groups, uint64_t* bytes_out) {
    if (!bytes_out || rows < 0 || n < 0 || k < 0 || groups < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!sizes_supported(rows, n, k, groups)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (codes_restored(n, k, groups)) {
        const int32_t rc = mega_moe_grouped_weight_workspace_bytes(rows, n, k, groups, bytes_out);
        *bytes_out += (uint64_t)rows * k * 2;
        return rc;
    }
    const int parts = codes_parts(rows, n, k, groups);
    *bytes_out = parts > 1 ? (uint64_t)parts * groups * n * k * 4 : 0;
    return MEGA_MOE_OK;
}

int32_t mega_moe_grouped_backward_weight_codes(const void* dy, const uint8_t* codes, const float* scales, const int32_t* offsets,
                                               void* dw, int64_t rows, int32_t n, int32_t k, int32_t groups, int32_t dtype,
                                               int32_t out_dtype, int32_t accumulate, void* workspace, uint64_t workspace_bytes,
                                               uint32_t* device_status, void* stream) {
    const int32_t rc = check_grouped(dy, dy, offsets, dw, rows, n, k, groups, dtype, device_status, true);
    if (rc) return rc;
    if (out_dtype != dtype && out_dtype != MEGA_MOE_FP32) return MEGA_MOE_ERR_UNSUPPORTED;
    if (accumulate && out_dtype != MEGA_MOE_FP32) return MEGA_MOE_ERR_UNSUPPORTED;
    if (weight_tiles(n, k, groups, 256) > (int64_t)1 << 21) return MEGA_MOE_ERR_UNSUPPORTED;
    if (rows > 0 && (!codes || ((uintptr_t)codes & 7u) || !scales || ((uintptr_t)scales & 3u))) return MEGA_MOE_ERR_INVALID_ARG;
    if (codes_restored(n, k, groups)) {       // restored behind the parts of the sum, then the product of 16-bit rows
        uint64_t need = 0;
        mega_moe_grouped_weight_workspace_bytes(rows, n, k, groups, &need);
        if (rows > 0 && !aligned16(workspace)) return MEGA_MOE_ERR_INVALID_ARG;
        if (workspace_bytes < need + (uint64_t)rows * k * 2) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
        void* x = static_cast<char*>(workspace) + need;
        if (mega_moe_dequantize_rows(codes, scales, x, rows, k, dtype, stream) != MEGA_MOE_OK) return MEGA_MOE_ERR_HIP;
        return mega_moe_grouped_backward_weight(dy, x, offsets, dw, rows, n, k, groups, dtype, out_dtype, accumulate, workspace, need,
                                                device_status, stream);
    }
    const int parts = codes_parts(rows, n, k, groups);
    if (parts > 1) {
        if (!aligned16(workspace)) return MEGA_MOE_ERR_INVALID_ARG;
        if (workspace_bytes < (uint64_t)parts * groups * n * k * 4) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    const CodesArgs a{{static_cast<const uint16_t*>(dy), nullptr, dw, offsets, device_status, (int)rows, n, k, groups, accumulate != 0, parts},
                      codes, scales};
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (out_dtype == MEGA_MOE_FP32)
        e = dtype == MEGA_MOE_BF16 ? launch_codes<Bf16, true>(a, workspace, st) : launch_codes<Fp16, true>(a, workspace, st);
    else
        e = dtype == MEGA_MOE_BF16 ? launch_codes<Bf16, false>(a, workspace, st) : launch_codes<Fp16, false>(a, workspace, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
