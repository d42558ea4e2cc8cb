// Products grouped by expert with ragged rows, and their gradients (include/mega_moe_ops.h):
//   forward          y[m]  = x[m] w[e]^T      P = x rows (KC),  Q = w rows (KC),   contraction k
//   backward_rows    dx[m] = dy[m] w[e]       P = dy rows (KC), Q = w columns (KS), contraction n
//   backward_weight  dw[e] = dy_e^T x_e       P = dy columns (KS), Q = x columns (KS), contraction rows
// The row-major weights are read as they are in all three: where the contraction runs down the memory rows
// the fragments are transposed on their way out of LDS.
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
};

// forward / backward_rows: one BM x BN tile of a group's rows per work-group
template <class T, bool kBackward, int BM, int BN, int WM, int WN, int NST>
__global__ __launch_bounds__(WM * WN * 64) void grouped_rows_kernel(GroupedArgs a) {
    using L = TileLoop<T, false, kBackward, BM, BN, WM, WN, NST>;
    __shared__ __align__(1024) uint8_t smem[L::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cols = kBackward ? a.k : a.n, depth = kBackward ? a.n : a.k;
    const TileMap<BM> map(a.off, a.groups, a.rows, (cols + BN - 1) / BN, 8, lane, blockIdx.x ? nullptr : a.status);
    const int tile = xcd_tile(blockIdx.x, map.total);
    if (tile < 0) return;
    const TileAt w = map.at(tile, lane);
    if (w.g < 0) return;
    const int m0 = w.mt * BM, q0 = w.nt * BN;
    const KcTile<BM, L::kWaves> P(a.p + (size_t)(w.lo + m0) * depth, w.cnt - m0, depth, depth, wave, lane);
    const uint16_t* wg = a.q + (size_t)w.g * a.n * a.k;
    f32x4 acc[L::QI][L::MI];
    const int steps = (depth + kStepK - 1) / kStepK;
    if constexpr (kBackward) {
        const KsTile<BN, L::kWaves> Q(wg, q0, a.k, a.n, wave, lane);
        L::run(P, Q, steps, smem, wave, lane, acc);
    } else {
        const KcTile<BN, L::kWaves> Q(wg + (size_t)q0 * a.k, a.n - q0, a.k, a.k, wave, lane);
        L::run(P, Q, steps, smem, wave, lane, acc);
    }
    const int wm = wave / WN, wn = wave % WN;
    uint16_t* out = static_cast<uint16_t*>(a.out);
#pragma unroll
    for (int j = 0; j < L::MI; ++j) {
        const int m = m0 + (wm * L::MI + j) * 16 + (lane & 15);
        uint16_t* row = out + (size_t)(w.lo + m) * cols;
#pragma unroll
        for (int i = 0; i < L::QI; ++i) {
            const int c = q0 + (wn * L::QI + i) * 16 + (lane >> 4) * 4;
            const f32x4 v = acc[i][j];
            if (m < w.cnt && c < cols)
                *reinterpret_cast<u32x2*>(row + c) = u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
        }
    }
}

// backward_weight: one BM x BN tile of dw[e] per work-group
template <class T, bool kFp32, int BM, int BN, int WM, int WN, int NST>
__global__ __launch_bounds__(WM * WN * 64) void grouped_weight_kernel(GroupedArgs a) {
    using L = TileLoop<T, true, true, BM, BN, WM, WN, NST>;
    __shared__ __align__(1024) uint8_t smem[L::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ntm = (a.n + BM - 1) / BM, ntq = (a.k + BN - 1) / BN;
    const int tile = xcd_tile(blockIdx.x, a.groups * ntm * ntq);
    if (tile < 0) return;
    const int g = tile / (ntm * ntq), li = tile - g * ntm * ntq;
    // bands of 8 row tiles, as the row products have bands of column tiles
    const int band = li / (8 * ntq), in = li - band * 8 * ntq, width = min(8, ntm - band * 8);
    const int qt = in / width, m0 = (band * 8 + in - qt * width) * BM, q0 = qt * BN;
    int lo, cnt;
    bool bad = false;
    group_rows(a.off, g, a.rows, lo, cnt, bad);
    lo = __builtin_amdgcn_readfirstlane(lo);
    cnt = __builtin_amdgcn_readfirstlane(cnt);
    if (bad && li == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, MEGA_MOE_STATUS_BAD_LAYOUT);
    f32x4 acc[L::QI][L::MI];
    const KsTile<BM, L::kWaves> P(a.p + (size_t)lo * a.n, m0, a.n, cnt, wave, lane);
    const KsTile<BN, L::kWaves> Q(a.q + (size_t)lo * a.k, q0, a.k, cnt, wave, lane);
    if (cnt == 0 && a.accumulate) return;
    L::run(P, Q, (cnt + kStepK - 1) / kStepK, smem, wave, lane, acc);
    const int wm = wave / WN, wn = wave % WN;
#pragma unroll
    for (int j = 0; j < L::MI; ++j) {
        const int m = m0 + (wm * L::MI + j) * 16 + (lane & 15);
        const size_t row = ((size_t)g * a.n + m) * a.k;
#pragma unroll
        for (int i = 0; i < L::QI; ++i) {
            const int c = q0 + (wn * L::QI + i) * 16 + (lane >> 4) * 4;
            if (m >= a.n || c >= a.k) continue;
            f32x4 v = acc[i][j];
            if constexpr (kFp32) {
                f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + row + c);
                if (a.accumulate) v += *o;
                *o = v;
            } else {
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + row + c) =
                    u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
            }
        }
    }
}

bool aligned16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }

int32_t check_grouped(const void* p, const void* q, const int32_t* off, const void* out, int64_t rows, int32_t n,
                      int32_t k, int32_t groups, int32_t dtype, const uint32_t* status, bool weight) {
    if (rows < 0 || n < 0 || k < 0 || groups < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (rows > MEGA_MOE_MAX_GROUP_ROWS || n < 8 || n > MEGA_MOE_MAX_GROUP_COLS || n % 8 || k < 8 ||
        k > MEGA_MOE_MAX_GROUP_COLS || k % 8 || groups < 1 || groups > MEGA_MOE_MAX_LOCAL_EXPERTS ||
        (dtype != MEGA_MOE_BF16 && dtype != MEGA_MOE_FP16))
        return MEGA_MOE_ERR_UNSUPPORTED;
    if (!off || ((uintptr_t)off & 3u) || ((uintptr_t)status & 3u)) return MEGA_MOE_ERR_INVALID_ARG;
    const bool any = rows > 0;
    if ((any && !aligned16(p)) || ((any || !weight) && !aligned16(q)) || ((any || weight) && !aligned16(out)))
        return MEGA_MOE_ERR_INVALID_ARG;
    return MEGA_MOE_OK;
}

template <class T, bool kBackward>
hipError_t launch_rows(const GroupedArgs& a, hipStream_t st) {
    constexpr int BM = 128, BN = 128;
    const int64_t tiles = ((int64_t)a.rows / BM + min((int64_t)a.groups, (int64_t)a.rows)) *
                          (((kBackward ? a.k : a.n) + BN - 1) / BN);
    hipLaunchKernelGGL((grouped_rows_kernel<T, kBackward, BM, BN, 2, 2, 2>), dim3((uint32_t)((tiles + 7) / 8 * 8)),
                       dim3(256), 0, st, a);
    return hipGetLastError();
}

template <class T, bool kFp32>
hipError_t launch_weight(const GroupedArgs& a, hipStream_t st) {
    constexpr int BM = 128, BN = 128;
    const int64_t tiles = (int64_t)a.groups * ((a.n + BM - 1) / BM) * ((a.k + BN - 1) / BN);
    hipLaunchKernelGGL((grouped_weight_kernel<T, kFp32, BM, BN, 2, 2, 2>), dim3((uint32_t)((tiles + 7) / 8 * 8)),
                       dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int32_t mega_moe_grouped_forward(const void* x, const void* w, const int32_t* offsets, void* y, int64_t rows, int32_t n,
                                 int32_t k, int32_t groups, int32_t dtype, uint32_t* device_status, void* stream) {
    const int32_t rc = check_grouped(x, w, offsets, y, rows, n, k, groups, dtype, device_status, false);
    if (rc || rows == 0) return rc;
    const GroupedArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), y, offsets, device_status,
                        (int)rows, n, k, groups, 0};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == MEGA_MOE_BF16 ? launch_rows<Bf16, false>(a, st) : launch_rows<Fp16, false>(a, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_grouped_backward_rows(const void* dy, const void* w, const int32_t* offsets, void* dx, int64_t rows,
                                       int32_t n, int32_t k, int32_t groups, int32_t dtype, uint32_t* device_status,
                                       void* stream) {
    const int32_t rc = check_grouped(dy, w, offsets, dx, rows, n, k, groups, dtype, device_status, false);
    if (rc || rows == 0) return rc;
    const GroupedArgs a{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(w), dx, offsets, device_status,
                        (int)rows, n, k, groups, 0};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == MEGA_MOE_BF16 ? launch_rows<Bf16, true>(a, st) : launch_rows<Fp16, true>(a, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_grouped_backward_weight(const void* dy, const void* x, const int32_t* offsets, void* dw, int64_t rows,
                                         int32_t n, int32_t k, int32_t groups, int32_t dtype, int32_t out_dtype,
                                         int32_t accumulate, uint32_t* device_status, void* stream) {
    const int32_t rc = check_grouped(dy, x, offsets, dw, rows, n, k, groups, dtype, device_status, true);
    if (rc) return rc;
    if (out_dtype != dtype && out_dtype != MEGA_MOE_FP32) return MEGA_MOE_ERR_UNSUPPORTED;
    if (accumulate && out_dtype != MEGA_MOE_FP32) return MEGA_MOE_ERR_UNSUPPORTED;
    // 32-bit tile numbers, and a launch of fewer than 2^32 threads
    if ((int64_t)groups * ((n + 127) / 128) * ((k + 127) / 128) > (int64_t)1 << 22) return MEGA_MOE_ERR_UNSUPPORTED;
    const GroupedArgs a{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(x), dw, offsets, device_status,
                        (int)rows, n, k, groups, accumulate != 0};
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (out_dtype == MEGA_MOE_FP32)
        e = dtype == MEGA_MOE_BF16 ? launch_weight<Bf16, true>(a, st) : launch_weight<Fp16, true>(a, st);
    else
        e = dtype == MEGA_MOE_BF16 ? launch_weight<Bf16, false>(a, st) : launch_weight<Fp16, false>(a, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
