// Activations in 8 bits and SwiGLU between the experts' products (include/mega_moe_ops.h):
//   quantize / dequantize  rows to codes and scales (row_io.h), and back
//   swiglu                 act = g / (1 + exp(-g)) u of a gate_up row (g, u), keeping the row in 8 bits on the way
//   swiglu_backward        s = 1 / (1 + exp(-g)):  dg = dact u s (1 + g (1 - s)), du = dact g s, and act again
// Elementwise: each pass reads and writes every byte once.  16 lanes take one block of 128 columns, 8 values a lane.
// exp and the reciprocal are the hardware's, a few 2^-24 relative (the product g log2 e adds |g| 2^-24): far below the
// 16-bit outputs' half steps of 2^-9 and 2^-12.
//
// Bound by memory.  Measured, bf16, 32768 x 2048: swiglu 58 us (403 MB, 6.9 TB/s), keeping its input 85 (541 MB, 6.4), the
// gradient from codes with act 104 (675 MB, 6.5); 1024 x 2048: 3.7 us.  32768 x 7168: quantize 119 us (712 MB, 6.0), restored 105
// (6.8); 8192 x 4096, in the last-level cache: 15 and 15.
#include "row_io.h"

namespace mm {
namespace {

// The blocks of 128 columns of many rows, dealt out to groups of 16 lanes: block b of row r, then the one `groups` further on.
struct Walk {
    int64_t row;
    int block, step_block;
    int64_t step_row;
    int blocks;
    __device__ __forceinline__ Walk(int n, int64_t first) {
        const int64_t groups = (int64_t)gridDim.x * 16, at = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
        blocks = n;
        row = first + at / n;
        block = (int)(at % n);
        step_row = groups / n;
        step_block = (int)(groups % n);
    }
    __device__ __forceinline__ void next() {
        row += step_row;
        block += step_block;
        if (block >= blocks) {
            block -= blocks;
            ++row;
        }
    }
};

__device__ __forceinline__ void keep(uint8_t* codes, float* scales, int64_t row, int block, int blocks, int cols, int c, float (&v)[8]) {
    const Scale s(max16(largest(v)));
    s.store<false>(codes, (size_t)row * cols + c, cols - c, v);
    if ((threadIdx.x & 15) == 0) scales[(size_t)row * blocks + block] = s.scale;
}

template <class T, bool kOnce>
__global__ __launch_bounds__(256) void quantize_kernel(const void* x, uint8_t* codes, float* scales, int rows, int cols) {
    for (Walk w(scale_blocks(cols), 0); w.row < rows; w.next()) {
        const int c = w.block * kScaleCols + (threadIdx.x & 15) * 8;
        float v[8];
        Row8<T>::template load<kOnce>(x, (size_t)w.row * cols + c, cols - c).get(v);
        keep(codes, scales, w.row, w.block, w.blocks, cols, c, v);
    }
}

template <class T>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* codes, const float* scales, void* y, int rows, int cols) {
    for (Walk w(scale_blocks(cols), 0); w.row < rows; w.next()) {
        const int c = w.block * kScaleCols + (threadIdx.x & 15) * 8;
        float v[8];
        Codes8::load<false>(codes, (size_t)w.row * cols + c, cols - c).get(scales[(size_t)w.row * w.blocks + w.block], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = restored<T>(v[i]);
        Row8<T>::store(y, (size_t)w.row * cols + c, cols - c, v);
    }
}
struct SwigluArgs {
    const void *dact, *gate_up;     // gate_up: values, or codes (backward)
    const float* in_scales;         // of codes
    void *act, *dgate_up;
    uint8_t* codes;                 // forward, may be null
    float* scales;
    const int32_t* offsets;         // may be null: all rows
    uint32_t* status;
    int groups, rows, inter;
};

// The rows of all groups together.
__device__ __forceinline__ void used_rows(const SwigluArgs& a, int& lo, int& hi) {
    lo = 0;
    hi = a.rows;
    if (!a.offsets) return;
    const int first = a.offsets[0], last = a.offsets[a.groups];
    lo = min(max(first, 0), a.rows);
    hi = max(min(last, a.rows), lo);
    if ((first < 0 || last < first || last > a.rows) && a.status && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(a.status, MEGA_MOE_STATUS_BAD_LAYOUT);
}

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

template <class T, bool kKeep, bool kOnce>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluArgs a) {
    int lo, hi;
    used_rows(a, lo, hi);
    for (Walk w(scale_blocks(a.inter), lo); w.row < hi; w.next()) {
        const int c = w.block * kScaleCols + (threadIdx.x & 15) * 8, n = a.inter - c;
        const size_t at = (size_t)w.row * a.inter;
        const Row8<T> gate = Row8<T>::template load<kOnce>(a.gate_up, 2 * at + c, n);
        const Row8<T> up = Row8<T>::template load<kOnce>(a.gate_up, 2 * at + a.inter + c, n);
        float g[8], u[8], y[8];
        gate.get(g);
        up.get(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = g[i] * sigmoid(g[i]) * u[i];
        Row8<T>::store(a.act, at + c, n, y);
        if constexpr (kKeep) {      // gate and up are kept as rows of their own
            keep(a.codes, a.scales, 2 * w.row, w.block, w.blocks, a.inter, c, g);
            keep(a.codes, a.scales, 2 * w.row + 1, w.block, w.blocks, a.inter, c, u);
        }
    }
}

template <class T, bool kCodes>
__global__ __launch_bounds__(256) void swiglu_grad_kernel(SwigluArgs a) {
    int lo, hi;
    used_rows(a, lo, hi);
    for (Walk w(scale_blocks(a.inter), lo); w.row < hi; w.next()) {
        const int c = w.block * kScaleCols + (threadIdx.x & 15) * 8, n = a.inter - c;
        const size_t at = (size_t)w.row * a.inter;
        const Row8<T> d8 = Row8<T>::load(a.dact, at + c, n);
        float d[8], g[8], u[8], y[8];
        if constexpr (kCodes) {
            const float* s = a.in_scales + (size_t)w.row * 2 * w.blocks + w.block;
            const Codes8 gate = Codes8::load<true>(a.gate_up, 2 * at + c, n), up = Codes8::load<true>(a.gate_up, 2 * at + a.inter + c, n);
            gate.get(s[0], g);
            up.get(s[w.blocks], u);
        } else {
            const Row8<T> gate = Row8<T>::load(a.gate_up, 2 * at + c, n), up = Row8<T>::load(a.gate_up, 2 * at + a.inter + c, n);
            gate.get(g);
            up.get(u);
        }
        d8.get(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = sigmoid(g[i]), gs = g[i] * s;
            y[i] = gs * u[i];
            u[i] = d[i] * u[i] * (s + gs * (1.0f - s));
            g[i] = d[i] * gs;
        }
        Row8<T>::store(a.dgate_up, 2 * at + c, n, u);
        Row8<T>::store(a.dgate_up, 2 * at + a.inter + c, n, g);
        if (a.act) Row8<T>::store(a.act, at + c, n, y);
    }
}

// 16 blocks of columns to a work-group at a time; at most 16 work-groups to a CU, which go on to further blocks.
dim3 walk_grid(int64_t rows, int cols) {
    const int64_t n = (rows * scale_blocks(cols) + 15) / 16;
    return dim3((uint32_t)(n < 4096 ? n : 4096));
}

template <class T>
hipError_t launch_quantize(const void* x, uint8_t* codes, float* scales, int rows, int cols, hipStream_t st) {
    const dim3 grid = walk_grid(rows, cols);
    if (beyond_cache((uint64_t)rows * cols * Row8<T>::kBytes))
        hipLaunchKernelGGL((quantize_kernel<T, true>), grid, dim3(256), 0, st, x, codes, scales, rows, cols);
    else
        hipLaunchKernelGGL((quantize_kernel<T, false>), grid, dim3(256), 0, st, x, codes, scales, rows, cols);
    return hipGetLastError();
}

template <class T>
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t st) {
    const dim3 grid = walk_grid(a.rows, a.inter);
    if (!a.codes) hipLaunchKernelGGL((swiglu_kernel<T, false, false>), grid, dim3(256), 0, st, a);
    else if (beyond_cache((uint64_t)a.rows * a.inter * 4)) hipLaunchKernelGGL((swiglu_kernel<T, true, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((swiglu_kernel<T, true, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

bool half(int32_t dtype) { return dtype == MEGA_MOE_BF16 || dtype == MEGA_MOE_FP16; }
bool element(const void* p, int32_t dtype) { return p && ((uintptr_t)p & (dtype == MEGA_MOE_FP32 ? 3u : 1u)) == 0; }
bool word(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }
bool rows_supported(int64_t rows, int32_t cols) {
    return rows <= MEGA_MOE_MAX_GROUP_ROWS && cols >= 1 && cols <= MEGA_MOE_MAX_GROUP_COLS;
}

int32_t check_swiglu(const SwigluArgs& a, int64_t rows, int32_t dtype) {
    if (rows < 0 || a.inter < 0 || a.groups < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!rows_supported(rows, a.inter) || !half(dtype)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (a.offsets && (a.groups < 1 || a.groups > MEGA_MOE_MAX_LOCAL_EXPERTS)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (((uintptr_t)a.offsets & 3u) || ((uintptr_t)a.status & 3u)) return MEGA_MOE_ERR_INVALID_ARG;
    return MEGA_MOE_OK;
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int32_t mega_moe_quantize_rows(const void* x, uint8_t* codes, float* scales, int64_t rows, int32_t cols, int32_t dtype, void* stream) {
    if (rows < 0 || cols < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!rows_supported(rows, cols) || (!half(dtype) && dtype != MEGA_MOE_FP32)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MEGA_MOE_OK;
    if (!element(x, dtype) || !codes || !word(scales)) return MEGA_MOE_ERR_INVALID_ARG;
    hipError_t e;
    if (dtype == MEGA_MOE_BF16) e = launch_quantize<Bf16>(x, codes, scales, (int)rows, cols, static_cast<hipStream_t>(stream));
    else if (dtype == MEGA_MOE_FP16) e = launch_quantize<Fp16>(x, codes, scales, (int)rows, cols, static_cast<hipStream_t>(stream));
    else e = launch_quantize<Fp32>(x, codes, scales, (int)rows, cols, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_dequantize_rows(const uint8_t* codes, const float* scales, void* y, int64_t rows, int32_t cols, int32_t dtype, void* stream) {
    if (rows < 0 || cols < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!rows_supported(rows, cols) || (!half(dtype) && dtype != MEGA_MOE_FP32)) return MEGA_MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MEGA_MOE_OK;
    if (!element(y, dtype) || !codes || !word(scales)) return MEGA_MOE_ERR_INVALID_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 grid = walk_grid(rows, cols);
    if (dtype == MEGA_MOE_BF16) hipLaunchKernelGGL((dequantize_kernel<Bf16>), grid, dim3(256), 0, st, codes, scales, y, (int)rows, cols);
    else if (dtype == MEGA_MOE_FP16) hipLaunchKernelGGL((dequantize_kernel<Fp16>), grid, dim3(256), 0, st, codes, scales, y, (int)rows, cols);
    else hipLaunchKernelGGL((dequantize_kernel<Fp32>), grid, dim3(256), 0, st, codes, scales, y, (int)rows, cols);
    return hipGetLastError() == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_swiglu(const void* gate_up, void* act, uint8_t* codes, float* scales, const int32_t* offsets, int32_t groups,
                        int64_t rows, int32_t inter, int32_t dtype, uint32_t* device_status, void* stream) {
    const SwigluArgs a{nullptr, gate_up, nullptr, act, nullptr, codes, scales, offsets, device_status, groups, (int)rows, inter};
    const int32_t rc = check_swiglu(a, rows, dtype);
    if (rc || rows == 0) return rc;
    if (!element(gate_up, dtype) || !element(act, dtype) || (codes != nullptr) != (scales != nullptr) || ((uintptr_t)scales & 3u))
        return MEGA_MOE_ERR_INVALID_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == MEGA_MOE_BF16 ? launch_swiglu<Bf16>(a, st) : launch_swiglu<Fp16>(a, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_swiglu_backward(const void* dact, const void* gate_up, const float* scales, void* dgate_up, void* act,
                                 const int32_t* offsets, int32_t groups, int64_t rows, int32_t inter, int32_t dtype,
                                 uint32_t* device_status, void* stream) {
    const SwigluArgs a{dact, gate_up, scales, act, dgate_up, nullptr, nullptr, offsets, device_status, groups, (int)rows, inter};
    const int32_t rc = check_swiglu(a, rows, dtype);
    if (rc || rows == 0) return rc;
    if (!element(dact, dtype) || !gate_up || (!scales && !element(gate_up, dtype)) || ((uintptr_t)scales & 3u) ||
        !element(dgate_up, dtype) || (act && !element(act, dtype)))
        return MEGA_MOE_ERR_INVALID_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const dim3 grid = walk_grid(rows, inter);
    if (dtype == MEGA_MOE_BF16) {
        if (scales) hipLaunchKernelGGL((swiglu_grad_kernel<Bf16, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((swiglu_grad_kernel<Bf16, false>), grid, dim3(256), 0, st, a);
    } else {
        if (scales) hipLaunchKernelGGL((swiglu_grad_kernel<Fp16, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((swiglu_grad_kernel<Fp16, false>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError() == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
