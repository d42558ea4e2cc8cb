// A projection shared by many requests that each bring a low-rank adapter (include/mega_moe_ops.h):
//   y[m] = x[m] w^T + scales[a] (x[m] a_a^T) b_a^T
// Two launches.  The first computes v[m] = scales[a] (x[m] a_a^T), a product grouped by request whose weight
// is the request's adapter, into the workspace.  The second computes the shared product tile by tile and adds
// v b_a^T to its accumulators before the one rounding of the output: the adapters cost rank / k of the shared
// product's operations and no pass over y.
//
// v is kept as two 16-bit numbers, hi = v rounded and lo = (v - hi) rounded, [rows][2][rank]: hi alone would add
// an error of half a step of the 16-bit type to every v; the second number takes it to 2^-17 (bf16) for twice
// the (few) operations of the second product.
#include "gemm_kernels.h"

namespace mm {
namespace {

struct AdapterArgs {
    const uint16_t *x, *w, *a, *b;
    const float* scales;
    const int32_t *off, *adapter;
    uint16_t *y, *v;
    uint32_t* status;
    int rows, n, k, rank, requests, adapters;
};

// The adapter of request r, or -1.
__device__ __forceinline__ int adapter_of(const AdapterArgs& g, int r) {
    const int i = g.adapter[r];
    return i >= 0 && i < g.adapters ? i : -1;
}

// Four values of v (columns c .. c+3 of row m) as hi and lo.
template <class T>
__device__ __forceinline__ void store_split(const AdapterArgs& g, int64_t m, int c, f32x4 v, float scale) {
    v *= scale;
    const u32x2 hi{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
    f32x4 rest{v[0] - T::low(hi[0]), v[1] - T::high(hi[0]), v[2] - T::low(hi[1]), v[3] - T::high(hi[1])};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (!(fabsf(rest[i]) < __builtin_inff())) rest[i] = 0.f;   // hi alone carries inf and NaN
    uint16_t* at = g.v + (size_t)m * 2 * g.rank + c;
    *reinterpret_cast<u32x2*>(at) = hi;
    *reinterpret_cast<u32x2*>(at + g.rank) = u32x2{T::pack(rest[0], rest[1]), T::pack(rest[2], rest[3])};
}

// v = scale * x a^T for one tile of a request's rows
template <class L, class T, int BM, int BN>
__global__ __launch_bounds__(L::kThreads) void adapter_down_kernel(AdapterArgs g) {
    __shared__ __align__(1024) uint8_t smem[L::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x == 0 && g.status)
        for (int r = threadIdx.x; r < g.requests; r += L::kThreads)
            if (g.adapter[r] < -1 || g.adapter[r] >= g.adapters) atomicOr(g.status, MEGA_MOE_STATUS_BAD_EXPERT_ID);
    const TileMap<BM> map(g.off, g.requests, g.rows, (g.rank + BN - 1) / BN, 8, lane, blockIdx.x ? nullptr : g.status);
    const int tile = xcd_tile(blockIdx.x, map.total);
    if (tile < 0) return;
    const TileAt t = map.at(tile, lane);
    if (t.g < 0) return;
    const int ad = __builtin_amdgcn_readfirstlane(adapter_of(g, t.g));
    if (ad < 0) return;
    const int m0 = t.mt * BM, c0 = t.nt * BN;
    const Operand P{g.x + (size_t)(t.lo + m0) * g.k, t.cnt - m0, g.k, g.k};
    const Operand Q{g.a + ((size_t)ad * g.rank + c0) * g.k, g.rank - c0, g.k, g.k};
    f32x4 acc[L::QI][L::MI];
    L::run(P, Q, smem, wave, lane, acc);
    const float scale = g.scales[ad];
#pragma unroll
    for (int j = 0; j < L::MI; ++j) {
        const int m = m0 + L::row(wave, j) + (lane & 15);
#pragma unroll
        for (int i = 0; i < L::QI; ++i) {
            const int c = c0 + L::col(wave, i) + (lane >> 4) * 4;
            if (m < t.cnt && c < g.rank) store_split<T>(g, t.lo + m, c, acc[i][j], scale);
        }
    }
}

// The first request that ends behind row m0 (requests sorted by row); all lanes take part.
__device__ __forceinline__ int first_request(const AdapterArgs& g, int m0, int lane) {
    int before = 0;
    for (int r0 = 0; r0 < g.requests; r0 += 64) {
        const uint64_t done = __ballot(r0 + lane < g.requests && g.off[r0 + lane + 1] <= m0);
        before += __popcll(done);
        if (done != ~0ull) break;
    }
    return before;
}

// 16 bytes of a row of values: columns c .. c+7, zeros from `cols` on.
__device__ __forceinline__ i32x4 row_chunk(const uint16_t* row, int c, int cols) {
    return c < cols ? *reinterpret_cast<const i32x4*>(row + c) : i32x4{0, 0, 0, 0};
}

// delta[i] = v b^T for the 16 rows of v from m (clamped to the last row) and this wave's column blocks of the
// tile from column q0
template <class T, class L>
__device__ __forceinline__ void adapter_delta(const AdapterArgs& g, int ad, int m, int q0, int wave, int lane,
                                              f32x4 (&delta)[L::QI]) {
    constexpr int QI = L::QI;
    const uint16_t* vrow = g.v + (size_t)min(m + (lane & 15), g.rows - 1) * 2 * g.rank;
    const uint16_t* b = g.b + (size_t)ad * g.n * g.rank;
#pragma unroll
    for (int i = 0; i < QI; ++i) delta[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < g.rank; c0 += 32) {
        const int c = c0 + (lane >> 4) * 8;
        const i32x4 hi = row_chunk(vrow, c, g.rank), lo = row_chunk(vrow + g.rank, c, g.rank);
#pragma unroll
        for (int i = 0; i < QI; ++i) {
            const int n = min(q0 + L::col(wave, i) + (lane & 15), g.n - 1);
            const i32x4 q = row_chunk(b + (size_t)n * g.rank, c, g.rank);
            delta[i] = T::mfma(q, hi, delta[i]);
            delta[i] = T::mfma(q, lo, delta[i]);
        }
    }
}

// y = x w^T + v b^T, one tile per work-group
template <class L, class T, int BM, int BN>
__global__ __launch_bounds__(L::kThreads) void adapter_up_kernel(AdapterArgs g) {
    __shared__ __align__(1024) uint8_t smem[L::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ntm = (g.rows + BM - 1) / BM, ntn = (g.n + BN - 1) / BN;
    const int tile = xcd_tile(blockIdx.x, ntm * ntn);
    if (tile < 0) return;
    const int band = tile / (ntm * 8), in = tile - band * ntm * 8, width = min(8, ntn - band * 8);
    const int m0 = in / width * BM, q0 = (band * 8 + in % width) * BN;
    const Operand P{g.x + (size_t)m0 * g.k, g.rows - m0, g.k, g.k}, Q{g.w + (size_t)q0 * g.k, g.n - q0, g.k, g.k};
    f32x4 acc[L::QI][L::MI];
    L::run(P, Q, smem, wave, lane, acc);
    // the requests that own rows of this tile, in order
    for (int r = first_request(g, m0, lane); r < g.requests; ++r) {
        int lo, cnt;
        bool bad = false;
        group_rows(g.off, r, g.rows, lo, cnt, bad);
        lo = __builtin_amdgcn_readfirstlane(lo);
        cnt = __builtin_amdgcn_readfirstlane(cnt);
        if (lo >= m0 + BM) break;
        const int ad = __builtin_amdgcn_readfirstlane(adapter_of(g, r));
        if (ad < 0) continue;
#pragma unroll
        for (int j = 0; j < L::MI; ++j) {
            const int mj = m0 + L::row(wave, j), m = mj + (lane & 15);
            if (lo >= mj + 16 || lo + cnt <= mj) continue;
            f32x4 delta[L::QI];
            adapter_delta<T, L>(g, ad, mj, q0, wave, lane, delta);
            // only this request's rows: another request's infinity must not reach a row by way of 0 * inf
            const bool mine = m >= lo && m < lo + cnt;
#pragma unroll
            for (int i = 0; i < L::QI; ++i) acc[i][j] += mine ? delta[i] : f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
    store_halves<L, T>(acc, g.y + (size_t)m0 * g.n + q0, g.rows - m0, g.n - q0, g.n, smem, wave, lane);
}

bool aligned(const void* p, uintptr_t to) { return p && ((uintptr_t)p & (to - 1)) == 0; }

template <class T>
hipError_t launch_adapter(const AdapterArgs& g, hipStream_t st) {
    if (g.requests > 0) {
        constexpr int BM = 64, BN = 64;
        const int64_t tiles = ((int64_t)g.rows / BM + min(g.requests, g.rows)) * ((g.rank + BN - 1) / BN);
        hipLaunchKernelGGL((adapter_down_kernel<TileLoop<T, false, false, BM, BN, 2, 2, 2>, T, BM, BN>), dim3((uint32_t)((tiles + 7) / 8 * 8)), dim3(256), 0,
                           st, g);
    }
    constexpr int BM = 128, BN = 128;
    const int64_t tiles = (int64_t)((g.rows + BM - 1) / BM) * ((g.n + BN - 1) / BN);
    hipLaunchKernelGGL((adapter_up_kernel<TileLoop<T, false, false, BM, BN, 2, 2, 2>, T, BM, BN>), dim3((uint32_t)((tiles + 7) / 8 * 8)), dim3(256), 0, st, g);
    return hipGetLastError();
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int32_t mega_moe_adapter_workspace_bytes(int64_t rows, int32_t rank, uint64_t* bytes_out) {
    if (!bytes_out || rows < 0 || rank < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (rows > MEGA_MOE_MAX_GROUP_ROWS || rank < 8 || rank > 256 || rank % 8) return MEGA_MOE_ERR_UNSUPPORTED;
    *bytes_out = (uint64_t)(rows > 0 ? rows : 1) * 2 * rank * 2;
    return MEGA_MOE_OK;
}

int32_t mega_moe_adapter_forward(const void* x, const void* w, const void* a, const void* b, const float* scales,
                                 const int32_t* offsets, const int32_t* adapter, void* y, int64_t rows, int32_t n,
                                 int32_t k, int32_t rank, int32_t requests, int32_t adapters, int32_t dtype,
                                 void* workspace, uint64_t workspace_bytes, uint32_t* device_status, void* stream) {
    if (n < 0 || k < 0 || requests < 0 || adapters < 0) return MEGA_MOE_ERR_INVALID_ARG;
    uint64_t need = 0;
    const int32_t rc = mega_moe_adapter_workspace_bytes(rows, rank, &need);
    if (rc) return rc;
    if (n < 8 || n > MEGA_MOE_MAX_GROUP_COLS || n % 8 || k < 8 || k > MEGA_MOE_MAX_GROUP_COLS || k % 8 ||
        requests > MEGA_MOE_MAX_REQUESTS || adapters < 1 || adapters > 65536 ||
        (dtype != MEGA_MOE_BF16 && dtype != MEGA_MOE_FP16))
        return MEGA_MOE_ERR_UNSUPPORTED;
    if (!aligned(w, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scales, 4) || !aligned(offsets, 4) ||
        (requests > 0 && !aligned(adapter, 4)) || !aligned(workspace, 16) || ((uintptr_t)device_status & 3u))
        return MEGA_MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!aligned(x, 16) || !aligned(y, 16))) return MEGA_MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    if (rows == 0) return MEGA_MOE_OK;
    const AdapterArgs g{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), static_cast<const uint16_t*>(a),
                        static_cast<const uint16_t*>(b), scales, offsets, adapter, static_cast<uint16_t*>(y),
                        static_cast<uint16_t*>(workspace), device_status, (int)rows, n, k, rank, requests, adapters};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == MEGA_MOE_BF16 ? launch_adapter<Bf16>(g, st) : launch_adapter<Fp16>(g, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
