// A projection shared by many requests that each bring a low-rank adapter (include/mega_moe_ops.h):
//   y[m] = x[m] w^T + scales[a] (x[m] a_a^T) b_a^T
//
// First launch, "down": u[m] = x[m] a_a^T, a product grouped by request whose weight is the request's adapter.  Its
// few tiles split the contraction between work-groups, and each part's fp32 sums go to the workspace.
//
// Many rows: the second launch computes the shared product tile by tile (gemm_kernels.h) and adds v b_a^T with
// v = scale * (sum of u's parts) to its accumulators before the one rounding of the output: the adapters cost
// rank / k of the shared product's operations and no pass over y.
//
// Few rows (up to kFewRows): a tile per work-group would leave most CUs without work, and the rows of many
// requests would wait for each other's adapters.  There the first launch also splits the shared product along the
// contraction, and the second ("join") has a wave for every 16 x 16 block of y, which adds up the parts and the
// adapters of its 16 rows.
//
// v enters the MFMA as two 16-bit numbers, hi = v rounded and lo = (v - hi) rounded: hi alone would add an
// error of half a step of the 16-bit type to every v; the second number takes it to 2^-16 (bf16) for twice the
// (few) operations of the second product.  fp16 has neither room for a large v nor bits for a small one: there the 32
// values of a row that one MFMA takes are multiplied by a power of two that brings the largest into 2^14 .. 2^15, and
// their fp32 sum by its inverse before it joins the others (8192 x 4096 x 7168, rank 64: 436 us against 435 without; at
// k 1024 and rank 256 181 against 174; 64 requests of a row 23.9 against 23.3).
//
// Measured, bf16.  64 requests of one row, rank 16, 4096 x 7168: 22 us for 68 MB (parts 16, join 7): bound by the
// weights' stream, which has 16 us to ramp up and drain, and the latency of two launches.  8192 rows of 12 requests,
// rank 64, 4096 x 7168: 404 us, 1210 TFLOP/s (down 25, bound by one read of x; up 380, bound by the MFMAs; with b's
// fragments read again for every 16 rows the whole took 420).  One row, rank 32, 7168 x 2048: 10 us replayed from
// a graph, 15 from the host, whose call takes as long.
#include <type_traits>

#include "gemm_kernels.h"

namespace mm {
namespace {

constexpr int kFewRows = 256;
constexpr int kMostParts = 8;          // of u

struct AdapterArgs {
    const uint16_t *x, *w, *a, *b;
    const float* scales;
    const int32_t *off, *adapter;
    uint16_t* y;
    uint32_t* status;
    float* u;          // [u_parts][rows][rank]
    float* part;       // few rows: [y_parts][rows][n]
    int32_t* of_row;   // few rows: [rows] adapter of every row, -1 for none
    int rows, n, k, rank, requests, adapters;
    int u_parts, u_steps, y_parts, y_steps;    // parts of the contraction and K steps of a part
};

// The adapter of request r, or -1.
__device__ __forceinline__ int adapter_of(const AdapterArgs& g, int r) {
    const int i = g.adapter[r];
    return i >= 0 && i < g.adapters ? i : -1;
}

// Part `s` of the contraction for an operand of `extent` rows of k values
__device__ __forceinline__ Operand part_of(const uint16_t* p, int extent, int k, int s, int steps) {
    const int k0 = s * steps * kStepK;
    return Operand{p + k0, extent, k, max(min(k - k0, steps * kStepK), 0)};
}

constexpr int kDownM = 64, kFewDownM = 32, kDownN = 64, kPartM = 64, kPartN = 128;
template <class T>
using DownLoop = TileLoop<T, false, false, kDownM, kDownN, 2, 2, 3>;
// A request of few rows is bound by the latency of one step after the other: four stages in flight
template <class T>
using FewDownLoop = TileLoop<T, false, false, kFewDownM, kDownN, 2, 2, 4>;
template <class T>
using PartLoop = TileLoop<T, false, false, kPartM, kPartN, 1, 4, 3>;

// One tile of u for one part of the contraction; block counts the down tiles times the parts.
template <class L>
__device__ __forceinline__ void down_tile(const AdapterArgs& g, int block, uint8_t* smem, int wave, int lane) {
    constexpr int kM = L::kRows;
    if (block == 0 && g.status)
        for (int r = threadIdx.x; r < g.requests; r += L::kThreads)
            if (g.adapter[r] < -1 || g.adapter[r] >= g.adapters) atomicOr(g.status, MEGA_MOE_STATUS_BAD_EXPERT_ID);
    const TileMap<kM> map(g.off, g.requests, g.rows, (g.rank + kDownN - 1) / kDownN, 8, lane,
                              block ? nullptr : g.status);
    const int part = block % g.u_parts, tile = block / g.u_parts;
    if (tile >= map.total) return;
    const TileAt t = map.at(tile, lane);
    if (t.g < 0) return;
    const int ad = __builtin_amdgcn_readfirstlane(adapter_of(g, t.g));
    if (ad < 0) return;
    const int m0 = t.mt * kM, c0 = t.nt * kDownN;
    const Operand P = part_of(g.x + (size_t)(t.lo + m0) * g.k, t.cnt - m0, g.k, part, g.u_steps);
    const Operand Q = part_of(g.a + ((size_t)ad * g.rank + c0) * g.k, g.rank - c0, g.k, part, g.u_steps);
    typename L::Acc acc[L::QI][L::MI];
    L::run(P, Q, smem, wave, lane, acc);
    float* u = g.u + ((size_t)part * g.rows + t.lo + m0) * g.rank + c0;
#pragma unroll
    for (int j = 0; j < L::MI; ++j)
#pragma unroll
        for (int i = 0; i < L::QI; ++i) {
            const int m = L::row(wave, j) + (lane & 15), c = L::col(wave, i) + (lane >> 4) * 4;
            if (m0 + m < t.cnt && c0 + c < g.rank) *reinterpret_cast<f32x4*>(u + (size_t)m * g.rank + c) = acc[i][j];
        }
}

template <class T>
__global__ __launch_bounds__(256) void adapter_down_kernel(AdapterArgs g) {
    static_assert(DownLoop<T>::kThreads == 256, "one launch");
    __shared__ __align__(1024) uint8_t smem[DownLoop<T>::kLds];
    down_tile<DownLoop<T>>(g, blockIdx.x, smem, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), threadIdx.x & 63);
}

// Few rows: work-groups 0 .. shared - 1 the parts of the shared product, then the rows' adapters, then the down tiles
template <class T>
__global__ __launch_bounds__(256) void adapter_parts_kernel(AdapterArgs g, int shared) {
    using L = PartLoop<T>;
    using Down = FewDownLoop<T>;
    static_assert(L::kThreads == 256 && Down::kThreads == 256, "one launch");
    __shared__ __align__(1024) uint8_t smem[L::kLds > Down::kLds ? L::kLds : Down::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int block = blockIdx.x;
    if (block >= shared) {
        block -= shared;
        if (block > 0) {
            down_tile<Down>(g, block - 1, smem, wave, lane);
            return;
        }
        for (int m = threadIdx.x; m < g.rows; m += 256) {
            // the last request that starts at or before row m and the first that ends behind it
            int lo = 0, hi = g.requests;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (g.off[mid + 1] > m) hi = mid;
                else lo = mid + 1;
            }
            g.of_row[m] = lo < g.requests && g.off[lo] <= m ? adapter_of(g, lo) : -1;
        }
        return;
    }
    // neighbouring work-groups of an XCD share the rows' part of the contraction
    const int ntm = (g.rows + kPartM - 1) / kPartM, ntn = (g.n + kPartN - 1) / kPartN;
    const int at = xcd_tile(block, ntm * ntn * g.y_parts);
    if (at < 0) return;
    const int part = at / (ntm * ntn), tile = at - part * ntm * ntn;
    const int m0 = tile % ntm * kPartM, q0 = tile / ntm * kPartN;
    const Operand P = part_of(g.x + (size_t)m0 * g.k, g.rows - m0, g.k, part, g.y_steps);
    const Operand Q = part_of(g.w + (size_t)q0 * g.k, g.n - q0, g.k, part, g.y_steps);
    typename L::Acc acc[L::QI][L::MI];
    L::run(P, Q, smem, wave, lane, acc);
    float* out = g.part + ((size_t)part * g.rows + m0) * g.n + q0;
#pragma unroll
    for (int j = 0; j < L::MI; ++j)
#pragma unroll
        for (int i = 0; i < L::QI; ++i) {
            const int m = L::row(wave, j) + (lane & 15), c = L::col(wave, i) + (lane >> 4) * 4;
            if (m0 + m < g.rows && q0 + c < g.n) *reinterpret_cast<f32x4*>(out + (size_t)m * g.n + c) = acc[i][j];
        }
}

// 16 bytes of a row of values: columns c .. c+7, zeros from `cols` on.
__device__ __forceinline__ i32x4 row_chunk(const uint16_t* row, int c, int cols) {
    return c < cols ? *reinterpret_cast<const i32x4*>(row + c) : i32x4{0, 0, 0, 0};
}

// The largest of v over the four lanes that hold a row's 32 values (l, l + 16, l + 32, l + 48); NaN does not count.
__device__ __forceinline__ float row_largest(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// scale * u[m][c .. c+7] (the parts added in their order) as hi and lo; zeros from column `rank` on.  Returns the factor
// of the product's sums (1 unless T::kNarrow).  All lanes take part.  kTogether: the
// loads of up to kMostParts parts go out before the first is needed (parts that do not exist repeat the last).
template <class T, bool kTogether>
__device__ __forceinline__ float low_rank_row(const AdapterArgs& g, int m, int c, float scale, i32x4& hi, i32x4& lo) {
    f32x4 v[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if (c < g.rank) {
        const float* u = g.u + (size_t)m * g.rank + c;
        if constexpr (kTogether) {
            f32x4 part[kMostParts][2];
#pragma unroll
            for (int s = 0; s < kMostParts; ++s) {
                const float* at = u + (size_t)min(s, g.u_parts - 1) * g.rows * g.rank;
                part[s][0] = *reinterpret_cast<const f32x4*>(at);
                part[s][1] = *reinterpret_cast<const f32x4*>(at + 4);
            }
#pragma unroll
            for (int s = 0; s < kMostParts; ++s)
                if (s < g.u_parts) {
                    v[0] += part[s][0];
                    v[1] += part[s][1];
                }
        } else {
            for (int s = 0; s < g.u_parts; ++s, u += (size_t)g.rows * g.rank) {
                v[0] += *reinterpret_cast<const f32x4*>(u);
                v[1] += *reinterpret_cast<const f32x4*>(u + 4);
            }
        }
    }
    float back = 1.f;
    if constexpr (T::kNarrow) {
        v[0] *= scale;
        v[1] *= scale;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i / 4][i % 4]));
        // biased exponent; the factors 2^(141 - e) and 2^(e - 141) are both normal numbers for it.  Of an infinite value
        // the factor is the largest number's, and of values below 2^-97 that of 2^-97
        const uint32_t e = min(max(__float_as_uint(row_largest(most)) >> 23, 30u), 254u);
        const float up = __uint_as_float((268 - e) << 23);
        back = __uint_as_float((e - 14) << 23);
        scale = up;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float a = v[h][2 * p] * scale, b = v[h][2 * p + 1] * scale;
            const uint32_t w = T::pack(a, b);
            float ra = a - T::low(w), rb = b - T::high(w);
            ra = fabsf(ra) < __builtin_inff() ? ra : 0.f;          // hi alone carries inf and NaN
            rb = fabsf(rb) < __builtin_inff() ? rb : 0.f;
            hi[h * 2 + p] = (int)w;
            lo[h * 2 + p] = (int)T::pack(ra, rb);
        }
    return back;
}

// sum + q (hi + lo), `back` from low_rank_row
template <class T>
__device__ __forceinline__ f32x4 add_low_rank(i32x4 q, i32x4 hi, i32x4 lo, float back, f32x4 sum) {
    if constexpr (T::kNarrow) return sum + back * T::mfma(q, lo, T::mfma(q, hi, f32x4{0.f, 0.f, 0.f, 0.f}));
    else return T::mfma(q, lo, T::mfma(q, hi, sum));
}

// Few rows: a wave per 16 x 16 block of y adds up the parts and its rows' adapters.  It is bound by the latency of its
// loads: the parts' are on their way while the adapters are looked up, and the b of kAtOnce adapters are read together.
// 16 where requests have few rows (64 rows with 24 adapters, rank 16: 6.4 us a launch, 7.2 with eight at a time, 9.8 with
// four and the parts first), 4 with half the registers where neighbouring rows share theirs.  kTogether for few blocks,
// which have no other waves to hide the reads of u behind: one row, rank 256, 4096 x 7168 23 us against 37 for the whole
// call; with 4096 blocks the registers cost more than that (256 rows of one request, rank 256: 84 against 50).
template <class T, int kAtOnce, bool kTogether>
__global__ __launch_bounds__(256) void adapter_join_kernel(AdapterArgs g) {
    const int lane = threadIdx.x & 63, col_blocks = (g.n + 15) / 16;
    const int block = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (block >= (g.rows + 15) / 16 * col_blocks) return;
    const int m0 = block / col_blocks * 16, n0 = block % col_blocks * 16;
    const int m = min(m0 + (lane & 15), g.rows - 1), n = n0 + (lane >> 4) * 4;
    const int ad = g.requests > 0 ? g.of_row[m] : -1;
    constexpr int kParts = 8;
    const float* p = g.part + (size_t)m * g.n + min(n, g.n - 4);
    f32x4 part[kParts];
#pragma unroll
    for (int s = 0; s < kParts; ++s) part[s] = *reinterpret_cast<const f32x4*>(p + (size_t)min(s, g.y_parts - 1) * g.rows * g.n);
    f32x4 sum{0.f, 0.f, 0.f, 0.f};
    uint32_t left = (uint32_t)__ballot(ad >= 0) & 0xFFFFu;        // rows whose adapter is still to be added
    const float scale = ad >= 0 ? g.scales[ad] : 0.f;
    const int nq = min(n0 + (lane & 15), g.n - 1), kq = (lane >> 4) * 8;
    while (left) {
        int id[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            id[i] = left ? __builtin_amdgcn_readlane(ad, __ffs(left) - 1) : -1;
            left &= ~(uint32_t)__ballot(ad == id[i]);
        }
        f32x4 delta[kAtOnce] = {};
        for (int c0 = 0; c0 < g.rank; c0 += 32) {
            const int c = c0 + kq;
            i32x4 q[kAtOnce], hi, lo;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                q[i] = row_chunk(g.b + ((size_t)max(id[i], 0) * g.n + nq) * g.rank, c, id[i] >= 0 ? g.rank : 0);
            // a row without an adapter has no u: its lanes stay at zero
            const float back = low_rank_row<T, kTogether>(g, m, ad >= 0 ? c : g.rank, scale, hi, lo);
            if constexpr (T::kNarrow) {
                // the factor is the row's, and so is the adapter: its sum is picked first (id -1 has zeros)
                f32x4 own{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const f32x4 d = T::mfma(q[i], lo, T::mfma(q[i], hi, f32x4{0.f, 0.f, 0.f, 0.f}));
                    own = ad == id[i] ? d : own;
                }
                sum += back * own;
            } else {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) delta[i] = T::mfma(q[i], lo, T::mfma(q[i], hi, delta[i]));
            }
        }
        // only its own rows: another request's infinity must not reach a row by way of 0 * inf
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (!T::kNarrow && id[i] >= 0) sum += ad == id[i] ? delta[i] : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    f32x4 shared = part[0];
#pragma unroll
    for (int s = 1; s < kParts; ++s) shared += s < g.y_parts ? part[s] : f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = kParts; s < g.y_parts; ++s) shared += *reinterpret_cast<const f32x4*>(p + (size_t)s * g.rows * g.n);
    sum += shared;
    if (m0 + (lane & 15) < g.rows && n < g.n)
        *reinterpret_cast<u32x2*>(g.y + (size_t)m * g.n + n) = u32x2{T::pack(sum[0], sum[1]), T::pack(sum[2], sum[3])};
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

// y = x w^T + v b^T for one tile.
template <class L, class T>
__device__ __forceinline__ void up_tile(const AdapterArgs& g, int m0, int q0, uint8_t* smem, int wave, int lane) {
    const Operand P{g.x + (size_t)m0 * g.k, g.rows - m0, g.k, g.k}, Q{g.w + (size_t)q0 * g.k, g.n - q0, g.k, g.k};
    typename L::Acc acc[L::QI][L::MI];
    L::run(P, Q, smem, wave, lane, acc);
    // the requests that own rows of this tile, in order
    for (int r = first_request(g, m0, lane); r < g.requests; ++r) {
        int lo, cnt;
        bool bad = false;
        group_rows(g.off, r, g.rows, lo, cnt, bad);
        lo = __builtin_amdgcn_readfirstlane(lo);
        cnt = __builtin_amdgcn_readfirstlane(cnt);
        if (lo >= m0 + L::kRows) break;
        const int ad = __builtin_amdgcn_readfirstlane(adapter_of(g, r));
        if (ad < 0) continue;
        const uint16_t* b = g.b + (size_t)ad * g.n * g.rank;
        const float scale = g.scales[ad];
        for (int c0 = 0; c0 < g.rank; c0 += 32) {
            const int c = c0 + (lane >> 4) * 8;
            i32x4 q[L::QI];
#pragma unroll
            for (int i = 0; i < L::QI; ++i) {
                const int n = min(q0 + L::col(wave, i) + (lane & 15), g.n - 1);
                q[i] = row_chunk(b + (size_t)n * g.rank, c, g.rank);
            }
#pragma unroll
            for (int j = 0; j < L::MI; ++j) {
                const int mj = m0 + L::row(wave, j), m = mj + (lane & 15);
                if (lo >= mj + 16 || lo + cnt <= mj) continue;
                // only this request's rows have its u, and only they get its sum: another request's infinity must
                // not reach a row by way of 0 * inf
                const bool mine = m >= lo && m < lo + cnt;
                i32x4 hi, lo16;
                const float back = low_rank_row<T, false>(g, min(m, g.rows - 1), mine ? c : g.rank, scale, hi, lo16);
#pragma unroll
                for (int i = 0; i < L::QI; ++i) {
                    const f32x4 sum = add_low_rank<T>(q[i], hi, lo16, back, acc[i][j]);
                    acc[i][j] = mine ? sum : acc[i][j];
                }
            }
        }
    }
    store_halves<L, T>(acc, g.y + (size_t)m0 * g.n + q0, g.rows - m0, g.n - q0, g.n, smem, wave, lane);
}

// H: a loop over half as many rows for the last row tile, as in the grouped products.
template <class L, class H, class T, int BM, int BN>
__global__ __launch_bounds__(L::kThreads) void adapter_up_kernel(AdapterArgs g) {
    static_assert(H::kThreads == L::kThreads, "one launch");
    __shared__ __align__(1024) uint8_t smem[L::kLds > H::kLds ? L::kLds : H::kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ntm = (g.rows + BM - 1) / BM, ntn = (g.n + BN - 1) / BN;
    const int tile = xcd_tile(blockIdx.x, ntm * ntn);
    if (tile < 0) return;
    // bands of 4 row tiles: the 32 tiles that an XCD runs at once are 4 x 8
    const int band = tile / (4 * ntn), in = tile - band * 4 * ntn, height = min(4, ntm - band * 4);
    const int m0 = (band * 4 + in % height) * BM, q0 = in / height * BN;
    if (!std::is_same<L, H>::value && g.rows - m0 <= BM / 2) up_tile<H, T>(g, m0, q0, smem, wave, lane);
    else up_tile<L, T>(g, m0, q0, smem, wave, lane);
}

bool aligned(const void* p, uintptr_t to) { return p && ((uintptr_t)p & (to - 1)) == 0; }

int clamp(int64_t v, int lo, int hi) { return (int)(v < lo ? lo : v > hi ? hi : v); }

// How the contraction is split, and the workspace: u's parts, then (few rows) y's parts and the rows' adapters.
struct Plan {
    bool few;
    int u_parts, u_steps, y_parts, y_steps;
    int64_t u_tiles, y_tiles;
    uint64_t part_at, row_at, total;
};
Plan plan_of(int rows, int n, int k, int rank, int requests) {
    Plan p{};
    const int steps = (k + kStepK - 1) / kStepK;
    p.few = rows <= kFewRows;
    p.u_tiles = requests > 0 ? ((int64_t)rows / (p.few ? kFewDownM : kDownM) + (requests < rows ? requests : rows)) * ((rank + kDownN - 1) / kDownN) : 0;
    p.y_tiles = (int64_t)((rows + kPartM - 1) / kPartM) * ((n + kPartN - 1) / kPartN);
    // at least four steps to a part, whose pipeline is three deep
    const int most = clamp(steps / 4, 1, kMostParts);
    const int64_t u_tiles = p.u_tiles > 0 ? p.u_tiles : 1;
    if (p.few) {
        // two work-groups to a CU at once, down tiles and shared tiles together; the longest part as short as that
        // allows, a step of either taking about as long, then the other's, then few parts to join (64 requests, 4096 x
        // 7168: 5 parts of u and 5 or 6 of y 24.4 us, 4 and 8 26.0, 6 and 4 25.6, 8 and 8 31.6)
        int least = 0;
        for (int y = 1; y <= 2 * most; ++y) {
            const int64_t left = 512 - p.y_tiles * y;
            if (y > 1 && left < p.u_tiles) break;
            const int u = clamp(left / u_tiles, 1, most), u_len = p.u_tiles > 0 ? (steps + u - 1) / u : 0, y_len = (steps + y - 1) / y;
            const int cost = 4 * (u_len > y_len ? u_len : y_len) + (u_len < y_len ? u_len : y_len) + y;
            if (y == 1 || cost < least) {
                least = cost;
                p.u_parts = u;
                p.y_parts = y;
            }
        }
    } else {
        p.u_parts = clamp(512 / u_tiles, 1, most);
        p.y_parts = 1;
    }
    const auto even = [&](int& parts, int& per) {
        per = (steps + parts - 1) / parts;
        parts = (steps + per - 1) / per;
    };
    even(p.u_parts, p.u_steps);
    even(p.y_parts, p.y_steps);
    const auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    p.part_at = up((uint64_t)p.u_parts * rows * rank * 4);
    p.row_at = p.part_at + (p.few ? up((uint64_t)p.y_parts * rows * n * 4) : 0);
    p.total = p.row_at + (p.few ? up((uint64_t)rows * 4) : 0) + 256;
    return p;
}

template <class L, class H, class T, int BM, int BN>
hipError_t launch_up(const AdapterArgs& g, hipStream_t st) {
    const int64_t tiles = (int64_t)((g.rows + BM - 1) / BM) * ((g.n + BN - 1) / BN);
    hipLaunchKernelGGL((adapter_up_kernel<L, H, T, BM, BN>), dim3((uint32_t)((tiles + 7) / 8 * 8)), dim3(L::kThreads), 0, st, g);
    return hipGetLastError();
}

template <class T>
hipError_t launch_adapter(const AdapterArgs& g, const Plan& p, hipStream_t st) {
    if (p.few) {
        const int shared = (int)((p.y_tiles * p.y_parts + 7) / 8 * 8);
        hipLaunchKernelGGL((adapter_parts_kernel<T>), dim3((uint32_t)(shared + 1 + p.u_tiles * p.u_parts)), dim3(256), 0, st, g,
                           shared);
        const int blocks = (g.rows + 15) / 16 * ((g.n + 15) / 16);
        const auto join = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((blocks + 3) / 4), dim3(256), 0, st, g); };
        if (g.requests > 4 && g.rows < 4 * g.requests) join(adapter_join_kernel<T, 16, false>);
        else if (blocks <= 512) join(adapter_join_kernel<T, 4, true>);
        else join(adapter_join_kernel<T, 4, false>);
        return hipGetLastError();
    }
    if (p.u_tiles > 0)
        hipLaunchKernelGGL((adapter_down_kernel<T>), dim3((uint32_t)(p.u_tiles * p.u_parts)), dim3(256), 0, st, g);
    using Wide = TileLoop<T, false, false, 128, 256, 2, 4, 3>;
    using Mid = TileLoop<T, false, false, 64, 128, 1, 4, 3>;
    using Square = TileLoop<T, false, false, 128, 128, 2, 4, 4>;
    switch (pick_row_shape(g.rows, g.n, g.k, 1, kShape64 + 1)) {
        case kShape256: return launch_up<QuadLoop<T, false, false, 256, 256, 4, 2>, Wide, T, 256, 256>(g, st);
        case kShape128: return launch_up<Wide, TileLoop<T, false, false, 64, 256, 1, 8, 3>, T, 128, 256>(g, st);
        case kShapeSquare: return launch_up<Square, TileLoop<T, false, false, 64, 128, 2, 4, 6>, T, 128, 128>(g, st);
        default: return launch_up<Mid, Mid, T, 64, 128>(g, st);
    }
}

int32_t check_sizes(int64_t rows, int32_t n, int32_t k, int32_t rank, int32_t requests) {
    if (rows < 0 || n < 0 || k < 0 || rank < 0 || requests < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (rows > MEGA_MOE_MAX_GROUP_ROWS || n < 8 || n > MEGA_MOE_MAX_GROUP_COLS || n % 8 || k < 8 ||
        k > MEGA_MOE_MAX_GROUP_COLS || k % 8 || rank < 8 || rank > 256 || rank % 8 || requests > MEGA_MOE_MAX_REQUESTS)
        return MEGA_MOE_ERR_UNSUPPORTED;
    // a launch has fewer than 2^32 threads
    if ((rows / 64 + 1) * ((n + 127) / 128) > (int64_t)1 << 23) return MEGA_MOE_ERR_UNSUPPORTED;
    return MEGA_MOE_OK;
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int32_t mega_moe_adapter_workspace_bytes(int64_t rows, int32_t n, int32_t k, int32_t rank, int32_t requests,
                                         uint64_t* bytes_out) {
    if (!bytes_out) return MEGA_MOE_ERR_INVALID_ARG;
    const int32_t rc = check_sizes(rows, n, k, rank, requests);
    if (rc) return rc;
    *bytes_out = plan_of((int)rows, n, k, rank, requests).total;
    return MEGA_MOE_OK;
}

int32_t mega_moe_adapter_forward(const void* x, const void* w, const void* a, const void* b, const float* scales,
                                 const int32_t* offsets, const int32_t* adapter, void* y, int64_t rows, int32_t n,
                                 int32_t k, int32_t rank, int32_t requests, int32_t adapters, int32_t dtype,
                                 void* workspace, uint64_t workspace_bytes, uint32_t* device_status, void* stream) {
    const int32_t rc = check_sizes(rows, n, k, rank, requests);
    if (rc) return rc;
    if (adapters < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (adapters < 1 || adapters > 65536 || (dtype != MEGA_MOE_BF16 && dtype != MEGA_MOE_FP16))
        return MEGA_MOE_ERR_UNSUPPORTED;
    if (!aligned(w, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(scales, 4) || !aligned(offsets, 4) ||
        (requests > 0 && !aligned(adapter, 4)) || !aligned(workspace, 16) || ((uintptr_t)device_status & 3u))
        return MEGA_MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!aligned(x, 16) || !aligned(y, 16))) return MEGA_MOE_ERR_INVALID_ARG;
    const Plan p = plan_of((int)rows, n, k, rank, requests);
    if (workspace_bytes < p.total) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    if (rows == 0) return MEGA_MOE_OK;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const AdapterArgs g{static_cast<const uint16_t*>(x),
                        static_cast<const uint16_t*>(w),
                        static_cast<const uint16_t*>(a),
                        static_cast<const uint16_t*>(b),
                        scales,
                        offsets,
                        adapter,
                        static_cast<uint16_t*>(y),
                        device_status,
                        reinterpret_cast<float*>(ws),
                        reinterpret_cast<float*>(ws + p.part_at),
                        reinterpret_cast<int32_t*>(ws + p.row_at),
                        (int)rows,
                        n,
                        k,
                        rank,
                        requests,
                        adapters,
                        p.u_parts,
                        p.u_steps,
                        p.y_parts,
                        p.y_steps};
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == MEGA_MOE_BF16 ? launch_adapter<Bf16>(g, p, st) : launch_adapter<Fp16>(g, p, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
