// Root-mean-square norm with the residual's addition, out in the input's type and in 8 bits with scales, and its
// gradient (include/mega_moe_ops.h):
//   forward    v = x + residual, r = 1 / sqrt(mean v^2 + eps), y = v r w
//   backward   r as above from h, n = h r, g = dy w:  dx = r (g - n mean(g n)) + dresidual,  dw = sum over rows of dy n
// One pass over memory: a row stays in the registers of its lanes between its reduction and its outputs.  All arithmetic
// is fp32 but the sums over a row, which are joined in fp64; y and the codes come from the unrounded sum v, each with its
// one rounding.
//
// Bound by memory.  Measured, bf16, 32768 x 7168: x, residual, h, y and codes 362 us (2.12 GB, 5.9 TB/s); x and y 193 us
// (4.9); the gradient with dresidual 354 us (1.88 GB, 5.3).  1024 x 7168 from an fp32 stream to codes: 17 us (4.8).  One row: 3.5 us,
// of which the launch is most.
#include <type_traits>

#include "row_io.h"

namespace mm {
namespace {

struct NormArgs {
    const void *x, *residual, *weight;   // x or residual may be null
    void *h, *y;                         // may be null
    uint8_t* codes;                      // may be null
    float* scales;
    int rows, hidden, weight_fp32;
    double mean, eps;                    // 1 / hidden
};

// Eight weights from column c on: fp32 or of type T.
template <class T>
__device__ __forceinline__ void weights8(const void* w, int fp32, int c, int n, float (&v)[8]) {
    if (fp32) Row8<Fp32>::load(w, c, n).get(v);
    else Row8<T>::load(w, c, n).get(v);
}

// Sums over the lanes of a row.  kLanes 16 or 64: within the wave.  0: the whole work-group, through LDS that alternates
// between two buffers from row to row, so that one barrier a row is enough: a buffer is written again only after the
// barrier of the row in between.  A lane adds its few values and the lanes are joined in fp64: r's error is that of every
// value of the row.
template <int kLanes, int kSums>
__device__ __forceinline__ void row_sums(double (&v)[kSums], double (*lds)[kSums], int turn) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] = kLanes == 16 ? sum16(v[i]) : sum64(v[i]);
    if constexpr (kLanes == 0) {
        const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
        double(*at)[kSums] = lds + turn * 16;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < kSums; ++i) at[wave][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSums; ++i) v[i] = 0.0;
        for (int w = 0; w < waves; ++w)
#pragma unroll
            for (int i = 0; i < kSums; ++i) v[i] += at[w][i];
    }
}
// 1 / sqrt(a), with one Newton step from the hardware's estimate; 0 and infinity, and NaN, as they come from it.
__device__ __forceinline__ double inverse_root(double a) {
    const double r = __builtin_amdgcn_rsq(a);
    return a > 0.0 && a < __builtin_inf() ? r * (1.5 - 0.5 * a * r * r) : r;
}

// y + rest, |rest| at most half a step of y, as y or, where y is even and there is a rest, the odd neighbour on its side:
// rounding it to fewer bits rounds y + rest.
__device__ __forceinline__ float odd(float y, float rest) {
    const uint32_t b = __float_as_uint(y);
    const uint32_t step = (int)(__float_as_uint(rest) ^ b) < 0 ? ~0u : 1u;
    return rest != 0.0f && !(b & 1u) && y != 0.0f ? __uint_as_float(b + step) : y;
}

// Where a lane stands: its row within the work-group, its place among the row's lanes, and their number.
template <int kLanes>
struct Place {
    int row, lane, lanes, rows;
    __device__ __forceinline__ Place() {
        lanes = kLanes ? kLanes : (int)blockDim.x;
        row = kLanes ? (int)threadIdx.x / kLanes : 0;
        lane = kLanes ? (int)threadIdx.x % kLanes : (int)threadIdx.x;
        rows = kLanes ? 256 / kLanes : 1;
    }
};

// T: x, y (and weight); R: residual, h.  A row's units of 8 columns go to its lanes in turn, kUnits to each.  kCodes: y in 8
// bits as well, or alone.
template <class T, class R, bool kCodes, int kLanes, int kUnits>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void rms_norm_kernel(NormArgs a) {
    __shared__ double lds[32][1];
    const Place<kLanes> p;
    int turn = 0;
    for (int row = blockIdx.x * p.rows + p.row; row < a.rows; row += gridDim.x * p.rows, turn ^= 1) {
        const size_t at = (size_t)row * a.hidden;
        Row8<T> x[kUnits];
        Row8<R> res[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = (u * p.lanes + p.lane) * 8;
            x[u] = Row8<T>::load(a.x, at + c, a.x ? a.hidden - c : 0);
            res[u] = Row8<R>::load(a.residual, at + c, a.residual ? a.hidden - c : 0);
        }
        float v[kUnits][8];
        typename std::conditional<kCodes, double, float>::type squares = 0;      // see below: codes ask for more of r
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = (u * p.lanes + p.lane) * 8;
            float r[8];
            x[u].get(v[u]);
            res[u].get(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[u][i] += r[i];
                squares += (decltype(squares))v[u][i] * v[u][i];
            }
            if (a.h) Row8<R>::store(a.h, at + c, a.hidden - c, v[u]);
        }
        double sum[1] = {squares};
        row_sums<kLanes>(sum, lds, turn);
        const double root = inverse_root(sum[0] * a.mean + a.eps);
        const float r = (float)root, lost = root < __builtin_inf() ? (float)(root - (double)r) : 0.f;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = (u * p.lanes + p.lane) * 8, n = a.hidden - c;
            float w[8];
            weights8<T>(a.weight, a.weight_fp32, c, n, w);
            if constexpr (!kCodes) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= r * w[i];
                if (a.y) Row8<T>::store(a.y, at + c, n, v[u]);
            } else {
                // For the codes a lane adds its squares in fp64 too, and what the products lose is added to them: y is within
                // half a step of fp32 of v r w, and what is left of it makes y odd, which the halves between two codes are
                // not.  So the codes are those of v r w, whatever v is in fp32: of 88 million values of bf16 rows none fell on
                // the other side of a half, 59 with fp32 throughout (32768 x 7168, y and codes: 362 us against 353).
                float rest[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float rw = r * w[i], less = v[u][i] * __builtin_fmaf(lost, w[i], __builtin_fmaf(r, w[i], -rw));
                    const float y = __builtin_fmaf(v[u][i], rw, less);
                    rest[i] = __builtin_fmaf(v[u][i], rw, -y) + less;
                    v[u][i] = y;
                }
                if (a.y) Row8<T>::store(a.y, at + c, n, v[u]);
                const Scale s(max16(largest(v[u])));
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = odd(v[u][i], rest[i]);
                s.template store<true>(a.codes, at + c, n, v[u]);
                if ((p.lane & 15) == 0 && n > 0) a.scales[(size_t)row * scale_blocks(a.hidden) + c / kScaleCols] = s.scale;
            }
        }
    }
}

struct NormGradArgs {
    const void *dy, *h, *weight, *dresidual;   // dresidual may be null
    const float* scales;                       // of h in codes
    void* dx;
    float* partial;                            // [gridDim.x][hidden]
    int rows, hidden, weight_fp32;
    double mean, eps;                          // 1 / hidden
};

// What a lane holds of a row as it is in memory.  T: dy; R: dresidual, and h unless kCodes.
template <class T, class R, bool kCodes, bool kOnce, int kUnits>
struct GradRow {
    Row8<T> dy[kUnits];
    typename std::conditional<kCodes, Codes8, Row8<R>>::type h[kUnits];
    float scale[kUnits];
    Row8<R> dres[kUnits];
    __device__ __forceinline__ void load(const NormGradArgs& a, int row, int lane, int lanes) {
        const size_t at = (size_t)row * a.hidden;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = (u * lanes + lane) * 8, n = row < a.rows ? a.hidden - c : 0;
            dy[u] = Row8<T>::template load<kOnce>(a.dy, at + c, n);
            h[u] = h[u].template load<kOnce>(a.h, at + c, n);
            scale[u] = 0.f;
            if (kCodes && n > 0) scale[u] = a.scales[(size_t)row * scale_blocks(a.hidden) + c / kScaleCols];
            dres[u] = Row8<R>::template load<kOnce>(a.dresidual, at + c, a.dresidual ? n : 0);
        }
    }
    // What was converted for the sums is converted again for dx: the fp32 values of both passes would take twice the registers.
    __device__ __forceinline__ void keep_packed() {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            dy[u].opaque();
            h[u].opaque();
        }
    }
    __device__ __forceinline__ void values(int u, float (&v)[8], float (&w)[8]) const {
        dy[u].get(v);
        if constexpr (kCodes) h[u].get(scale[u], w);
        else h[u].get(w);
    }
};

// T: dy (and weight); R: dresidual, dx, and h unless kCodes.  The next row is on its way while one is reduced and written.
template <class T, class R, bool kCodes, bool kOnce, int kLanes, int kUnits>
__global__ __launch_bounds__(kLanes ? 256 : 512) void rms_norm_grad_kernel(NormGradArgs a) {
    __shared__ double lds[32][2];
    const Place<kLanes> p;
    float dw[kUnits][8];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[u][i] = 0.f;
    int turn = 0, row = blockIdx.x * p.rows + p.row;
    const int step = gridDim.x * p.rows;
    // (four units a lane leave no registers for the next row)
    constexpr bool kAhead = kUnits <= 2;
    GradRow<T, R, kCodes, kOnce, kUnits> next;
    if (kAhead) next.load(a, row, p.lane, p.lanes);
    for (; row < a.rows; row += step, turn ^= 1) {
        const size_t at = (size_t)row * a.hidden;
        if (!kAhead) next.load(a, row, p.lane, p.lanes);
        GradRow<T, R, kCodes, kOnce, kUnits> here = next;
        if (kAhead) next.load(a, row + step, p.lane, p.lanes);
        float squares = 0.f, products = 0.f;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = (u * p.lanes + p.lane) * 8;
            float w[8], dy[8], h[8];
            weights8<T>(a.weight, a.weight_fp32, c, a.hidden - c, w);
            here.values(u, dy, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                squares += h[i] * h[i];
                products += dy[i] * w[i] * h[i];
            }
        }
        double sum[2] = {squares, products};
        row_sums<kLanes>(sum, lds, turn);
        const float r = (float)inverse_root(sum[0] * a.mean + a.eps), m = (float)(sum[1] * a.mean) * r;   // mean(g n)
        here.keep_packed();
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int c = (u * p.lanes + p.lane) * 8, n = a.hidden - c;
            float w[8], d[8], dy[8], h[8];
            weights8<T>(a.weight, a.weight_fp32, c, n, w);
            here.values(u, dy, h);
            here.dres[u].get(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float nv = h[i] * r;
                d[i] += r * (dy[i] * w[i] - nv * m);
                dw[u][i] += dy[i] * nv;
            }
            Row8<R>::store(a.dx, at + c, n, d);
        }
    }
    // one partial sum of dw per work-group: the rows of a wave, then the waves in their order
    if constexpr (kLanes != 0) {
        if constexpr (kLanes == 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[0][i] += __shfl_xor(dw[0][i], 16);
                dw[0][i] += __shfl_xor(dw[0][i], 32);
            }
        }
        __shared__ float waves[3][kUnits][8][kLanes];
        const int wave = threadIdx.x >> 6;
        if (wave > 0 && (int)(threadIdx.x & 63) < kLanes) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) waves[wave - 1][u][i][p.lane] = dw[u][i];
        }
        __syncthreads();
        if ((int)threadIdx.x >= kLanes) return;
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int w = 0; w < 3; ++w) dw[u][i] += waves[w][u][i][p.lane];
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int c = (u * p.lanes + p.lane) * 8;
        Row8<Fp32>::store(a.partial, (size_t)blockIdx.x * a.hidden + c, a.hidden - c, dw[u]);
    }
}

// dw = the work-groups' partial sums in their order: 32 columns x 32 runs of partial sums to a work-group
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* partial, float* dw, int parts, int hidden) {
    __shared__ float lds[32][33];
    const int col = threadIdx.x & 31, run = threadIdx.x >> 5, c = blockIdx.x * 32 + col, per = (parts + 31) / 32;
    float v = 0.f;
    if (c < hidden) {
        const int end = min(parts, (run + 1) * per);
#pragma unroll 8
        for (int i = run * per; i < end; ++i) v += partial[(size_t)i * hidden + c];
    }
    lds[run][col] = v;
    __syncthreads();
    if (run) return;
    for (int i = 1; i < 32; ++i) v += lds[i][col];
    if (c < hidden) dw[c] = v;
}

// ---------------------------------------------------------------- shapes
// The lanes of a row: 16 up to 128 columns, a wave up to 2048, else a work-group with as many waves as the units need.
struct RowShape8 {
    int lanes, units, threads, rows;    // rows: of a work-group at a time
};
RowShape8 row_shape(int hidden, int max_threads) {
    const int n = (hidden + 7) / 8;
    if (n <= 16) return {16, 1, 256, 16};
    if (n <= 64) return {64, 1, 256, 4};
    if (n <= 128) return {64, 2, 256, 4};
    if (n <= 256) return {64, 4, 256, 4};
    int units = 2;
    while ((n + units - 1) / units > max_threads) units *= 2;
    return {0, units, ((n + units - 1) / units + 63) / 64 * 64, 1};
}

// Work-groups of the gradient, which have a partial sum of dw each: those that are resident at once, 16 waves to a CU by the
// registers (32768 rows: 7168 columns, 7 waves: 374 us with 512, 423 with 256, 378 with 1024 and 416 with 2048; 4096
// columns, 4 waves: 223 with 512, 211 with 1024).
int grad_blocks(int64_t rows, int hidden) {
    const RowShape8 s = row_shape(hidden, 512);
    const int64_t n = (rows + s.rows - 1) / s.rows;
    const int64_t most = 256 * (16 / (s.threads / 64));
    return (int)(n < most ? n : most);
}

template <class T, class R, int kLanes, int kUnits>
hipError_t launch_norm_with(const NormArgs& a, const RowShape8& s, hipStream_t st) {
    const int64_t blocks = ((int64_t)a.rows + s.rows - 1) / s.rows;
    const dim3 grid((uint32_t)(blocks < (1 << 20) ? blocks : 1 << 20)), threads(s.threads);
    if (a.codes) hipLaunchKernelGGL((rms_norm_kernel<T, R, true, kLanes, kUnits>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((rms_norm_kernel<T, R, false, kLanes, kUnits>), grid, threads, 0, st, a);
    return hipGetLastError();
}
template <class T, class R>
hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
    const RowShape8 s = row_shape(a.hidden, 1024);
    if (s.lanes == 16) return launch_norm_with<T, R, 16, 1>(a, s, st);
    if (s.lanes == 64 && s.units == 1) return launch_norm_with<T, R, 64, 1>(a, s, st);
    if (s.lanes == 64) return s.units == 2 ? launch_norm_with<T, R, 64, 2>(a, s, st) : launch_norm_with<T, R, 64, 4>(a, s, st);
    return launch_norm_with<T, R, 0, 2>(a, s, st);
}

template <class T, class R, bool kCodes, int kLanes, int kUnits>
hipError_t launch_grad_with(const NormGradArgs& a, const RowShape8& s, hipStream_t st) {
    const dim3 grid((uint32_t)grad_blocks(a.rows, a.hidden)), threads(s.threads);
    const uint64_t each = (uint64_t)a.rows * a.hidden, bytes = each * (Row8<T>::kBytes + (kCodes ? 1 : Row8<R>::kBytes) + (a.dresidual ? Row8<R>::kBytes : 0));
    if (beyond_cache(bytes)) hipLaunchKernelGGL((rms_norm_grad_kernel<T, R, kCodes, true, kLanes, kUnits>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((rms_norm_grad_kernel<T, R, kCodes, false, kLanes, kUnits>), grid, threads, 0, st, a);
    return hipGetLastError();
}
template <class T, class R, bool kCodes>
hipError_t launch_grad(const NormGradArgs& a, hipStream_t st) {
    const RowShape8 s = row_shape(a.hidden, 512);
    if (s.lanes == 16) return launch_grad_with<T, R, kCodes, 16, 1>(a, s, st);
    if (s.lanes == 64 && s.units == 1) return launch_grad_with<T, R, kCodes, 64, 1>(a, s, st);
    if (s.lanes == 64) return s.units == 2 ? launch_grad_with<T, R, kCodes, 64, 2>(a, s, st) : launch_grad_with<T, R, kCodes, 64, 4>(a, s, st);
    return s.units == 2 ? launch_grad_with<T, R, kCodes, 0, 2>(a, s, st) : launch_grad_with<T, R, kCodes, 0, 4>(a, s, st);
}
template <bool kCodes>
hipError_t launch_grad_types(const NormGradArgs& a, int dtype, int residual_dtype, hipStream_t st) {
    if (dtype == MEGA_MOE_FP32) return launch_grad<Fp32, Fp32, kCodes>(a, st);
    if (dtype == MEGA_MOE_BF16)
        return residual_dtype == MEGA_MOE_FP32 ? launch_grad<Bf16, Fp32, kCodes>(a, st) : launch_grad<Bf16, Bf16, kCodes>(a, st);
    return residual_dtype == MEGA_MOE_FP32 ? launch_grad<Fp16, Fp32, kCodes>(a, st) : launch_grad<Fp16, Fp16, kCodes>(a, st);
}

// ---------------------------------------------------------------- checks
bool known(int32_t dtype) { return dtype == MEGA_MOE_BF16 || dtype == MEGA_MOE_FP16 || dtype == MEGA_MOE_FP32; }
bool aligned(const void* p, int32_t dtype) { return ((uintptr_t)p & (dtype == MEGA_MOE_FP32 ? 3u : 1u)) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool norm_supported(int64_t rows, int32_t hidden, float eps, int32_t dtype, int32_t residual_dtype, int32_t weight_dtype) {
    return rows <= MEGA_MOE_MAX_GROUP_ROWS && hidden >= 1 && hidden <= MEGA_MOE_MAX_NORM_COLS && eps >= 0.0f && eps < 3.4e38f &&
           known(dtype) && (residual_dtype == dtype || residual_dtype == MEGA_MOE_FP32) &&
           (weight_dtype == dtype || weight_dtype == MEGA_MOE_FP32);
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int32_t mega_moe_rms_norm(const void* x, const void* residual, const void* weight, void* h, void* y, uint8_t* codes, float* scales,
                          int64_t rows, int32_t hidden, float eps, int32_t dtype, int32_t residual_dtype, int32_t weight_dtype,
                          void* stream) {
    if (rows < 0 || hidden < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!norm_supported(rows, hidden, eps, dtype, residual_dtype, weight_dtype)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MEGA_MOE_OK;
    if (!weight || (!x && !residual) || (!y && !codes && !h) || (codes != nullptr) != (scales != nullptr)) return MEGA_MOE_ERR_INVALID_ARG;
    if (!aligned(x, dtype) || !aligned(residual, residual_dtype) || !aligned(weight, weight_dtype) || !aligned(h, residual_dtype) ||
        !aligned(y, dtype) || !aligned4(scales))
        return MEGA_MOE_ERR_INVALID_ARG;
    const NormArgs a{x, residual, weight, h, y, codes, scales, (int)rows, hidden, weight_dtype == MEGA_MOE_FP32, 1.0 / hidden, eps};
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (dtype == MEGA_MOE_FP32) e = launch_norm<Fp32, Fp32>(a, st);
    else if (dtype == MEGA_MOE_BF16)
        e = residual_dtype == MEGA_MOE_FP32 ? launch_norm<Bf16, Fp32>(a, st) : launch_norm<Bf16, Bf16>(a, st);
    else
        e = residual_dtype == MEGA_MOE_FP32 ? launch_norm<Fp16, Fp32>(a, st) : launch_norm<Fp16, Fp16>(a, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_norm_workspace_bytes(int64_t rows, int32_t hidden, uint64_t* bytes_out) {
    if (!bytes_out || rows < 0 || hidden < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!norm_supported(rows, hidden, 0.0f, MEGA_MOE_FP32, MEGA_MOE_FP32, MEGA_MOE_FP32)) return MEGA_MOE_ERR_UNSUPPORTED;
    *bytes_out = (uint64_t)grad_blocks(rows, hidden) * hidden * 4;
    return MEGA_MOE_OK;
}

int32_t mega_moe_rms_norm_backward(const void* dy, const void* h, const float* h_scales, const void* weight, const void* dresidual,
                                   void* dx, float* dweight, int64_t rows, int32_t hidden, float eps, int32_t dtype,
                                   int32_t residual_dtype, int32_t weight_dtype, void* workspace, uint64_t workspace_bytes, void* stream) {
    if (rows < 0 || hidden < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!norm_supported(rows, hidden, eps, dtype, residual_dtype, weight_dtype)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (!dweight || !aligned4(dweight)) return MEGA_MOE_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!dy || !h || !weight || !dx || !workspace) return MEGA_MOE_ERR_INVALID_ARG;
        if (!aligned(dy, dtype) || (!h_scales && !aligned(h, residual_dtype)) || !aligned4(h_scales) || !aligned(weight, weight_dtype) ||
            !aligned(dresidual, residual_dtype) || !aligned(dx, residual_dtype) || !aligned4(workspace))
            return MEGA_MOE_ERR_INVALID_ARG;
        if (workspace_bytes < (uint64_t)grad_blocks(rows, hidden) * hidden * 4) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int blocks = grad_blocks(rows, hidden);
    if (rows > 0) {
        const NormGradArgs a{dy, h, weight, dresidual, h_scales, dx, static_cast<float*>(workspace), (int)rows, hidden,
                             weight_dtype == MEGA_MOE_FP32, 1.0 / hidden, eps};
        const hipError_t e = h_scales ? launch_grad_types<true>(a, dtype, residual_dtype, st) : launch_grad_types<false>(a, dtype, residual_dtype, st);
        if (e != hipSuccess) return MEGA_MOE_ERR_HIP;
    }
    hipLaunchKernelGGL(norm_join_kernel, dim3((hidden + 31) / 32), dim3(1024), 0, st, static_cast<const float*>(workspace), dweight,
                       blocks, hidden);
    return hipGetLastError() == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
