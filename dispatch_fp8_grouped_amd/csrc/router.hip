// The router around the fused layer (include/mega_moe_ops.h): the choice and weights of each token's experts,
// the gradient of the weights, and the ordering of the chosen pairs by expert.
//
// Choice: one wave per token; lane l holds experts l*EPL .. l*EPL + EPL-1 (so the lowest lane of a tie holds
// the lowest expert).  An expert's rank becomes an unsigned key whose order is the rank's order, 0 for an
// expert that may not be chosen: 32 bits from the logit alone, 64 bits from the fp64 score + bias.  Each of the
// K rounds takes the wave's largest high word; only where several lanes share it do the low words decide.
//
// Scores are computed in fp64 (exp of the C library's device functions): two scores that differ in fp32
// logits then differ in rank, and the choice does not hang on a rounding of exp.
#include "gemm_tiles.h"

namespace mm {
namespace {

constexpr uint32_t kPairsPerWave = 256;      // pairs that one wave of the ordering ranks, 64 at a time
constexpr int kOneGroupPairs = 8192;         // up to here one work-group orders everything in one launch
constexpr int kOneGroupExperts = 512;       // 32 KB of counters

struct RouterArgs {
    const void* logits;
    const float* bias;
    int64_t* idx;
    float* weights;
    const float* dweights;
    void* dlogits;
    int64_t tokens;
    int E, K, G, kept, gtop, type;
    float scale;
    bool renorm;
};

// Element i of a tensor of MEGA_MOE_* type `type` (the same for the whole launch).
__device__ __forceinline__ float read_value(const void* p, int type, size_t i) {
    if (type == MEGA_MOE_FP32) return static_cast<const float*>(p)[i];
    if (type == MEGA_MOE_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
    return (float)static_cast<const _Float16*>(p)[i];
}
__device__ __forceinline__ void write_value(void* p, int type, size_t i, double v) {
    if (type == MEGA_MOE_FP32) static_cast<float*>(p)[i] = (float)v;
    else if (type == MEGA_MOE_BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16((float)v);
    else static_cast<_Float16*>(p)[i] = (_Float16)(float)v;
}

// This lane's EPL logits of a row of E; -inf past the row.  Where E is a multiple of EPL, every lane's
// values lie in the row or all behind it, and are aligned to their own size: one or a few wide loads.
template <int EPL, class V, class F>
__device__ __forceinline__ void read_lane(const V* row, int E, int lane, float (&x)[EPL], F value) {
    constexpr int kWide = EPL * (int)sizeof(V) < 16 ? EPL : 16 / (int)sizeof(V);
    struct __align__(kWide * sizeof(V)) Wide { V v[kWide]; };
    const int e0 = lane * EPL;
    if (E % EPL == 0) {
#pragma unroll
        for (int j = 0; j < EPL; j += kWide) {
            Wide w{};
            if (e0 < E) w = *reinterpret_cast<const Wide*>(row + e0 + j);
#pragma unroll
            for (int i = 0; i < kWide; ++i) x[j + i] = e0 < E ? value(w.v[i]) : -__builtin_inff();
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) x[j] = e0 + j < E ? value(row[e0 + j]) : -__builtin_inff();
    }
}
template <int EPL>
__device__ __forceinline__ void read_row(const void* p, int type, int64_t t, int E, int lane, float (&x)[EPL]) {
    const size_t at = (size_t)t * E;
    if (type == MEGA_MOE_FP32)
        read_lane(static_cast<const float*>(p) + at, E, lane, x, [](float v) { return v; });
    else if (type == MEGA_MOE_BF16)
        read_lane(static_cast<const uint16_t*>(p) + at, E, lane, x, [](uint16_t v) { return bf16_to_f32(v); });
    else
        read_lane(static_cast<const _Float16*>(p) + at, E, lane, x, [](_Float16 v) { return (float)v; });
}

// A masked logit is -inf or NaN; +inf counts as the largest fp32 number.
__device__ __forceinline__ bool is_masked(float x) { return !(x > -__builtin_inff()); }
__device__ __forceinline__ float clip_inf(float x) { return fminf(x, 3.402823466e38f); }

// Unsigned integers in the order of the numbers (no NaN); no number maps to 0.
__device__ __forceinline__ uint32_t order32(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);        // -0 ranks with +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order64(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
    return v;
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// A pair of largest values, merged
__device__ __forceinline__ void merge_top2(double& a, double& b, double c, double d) {
    const double hi = fmax(a, c), lo = fmin(a, c);
    b = fmax(lo, fmax(b, d));
    a = hi;
}

// kWide: 64-bit ranks (a bias is given); waves of a work-group take consecutive tokens.
template <int EPL, bool kSigmoid, bool kWide, bool kGroups, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void router_kernel(RouterArgs a) {
    __shared__ double values[kGroups ? WAVES : 1][kGroups ? EPL * 64 : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double none = -__builtin_inf();
    for (int64_t t = (int64_t)blockIdx.x * WAVES + wave; t < a.tokens; t += (int64_t)gridDim.x * WAVES) {
        float x[EPL];
        bool live[EPL];
        float top = -__builtin_inff();
        read_row<EPL>(a.logits, a.type, t, a.E, lane, x);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            live[j] = !is_masked(x[j]);
            x[j] = clip_inf(x[j]);
            if (live[j]) top = fmaxf(top, x[j]);
        }
        top = wave_max(top);                       // -inf where everything is masked
        // softmax needs its sum where the scores themselves enter the result; where they are divided by
        // the chosen ones' sum it cancels
        const bool by_score = kWide || (kGroups && a.gtop == 2);
        double total = 1.0;
        if (!kSigmoid && (by_score || !a.renorm)) {
            total = 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (live[j]) total += exp((double)x[j] - (double)top);
            total = wave_sum(total);
        }
        uint32_t hi[EPL], lo[kWide ? EPL : 1];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane * EPL + j;
            double rank = x[j], worth = x[j];
            if ((kWide || (kGroups && a.gtop == 2)) && live[j]) {
                const double s = kSigmoid ? sigmoid64(x[j]) : exp((double)x[j] - (double)top) / total;
                worth = s;
                if constexpr (kWide) {
                    worth = rank = s + (double)a.bias[e];
                    live[j] = rank > none;         // not -inf, not NaN
                }
            }
            if constexpr (kWide) {
                const uint64_t key = live[j] ? order64(rank) : 0;
                hi[j] = (uint32_t)(key >> 32);
                lo[j] = (uint32_t)key;
            } else {
                hi[j] = live[j] ? order32(x[j]) : 0;
            }
            if constexpr (kGroups) values[wave][e] = live[j] ? worth : none;
        }
        if constexpr (kGroups) {
            // L lanes per group (a power of two); group g's lanes are g*L .. g*L + L-1
            int L = 1;
            while (L * 2 * a.G <= 64) L *= 2;
            const int size = a.E / a.G, g = lane / L;
            double first = none, second = none;
            __builtin_amdgcn_wave_barrier();
            if (g < a.G)
                for (int i = lane % L; i < size; i += L) merge_top2(first, second, values[wave][g * size + i], none);
            for (int d = 1; d < L; d <<= 1) {
                const double c = __shfl_xor(first, d), e2 = __shfl_xor(second, d);
                merge_top2(first, second, c, e2);
            }
            // a group's worth: its best, or the sum of its two best where it has two
            double worth = first;
            if (a.gtop == 2 && second > none) worth += second;
            bool open = (lane % L) == 0 && g < a.G && first > none;
            uint64_t kept = 0;                     // bit of every kept group's first lane
            for (int r = 0; r < a.kept; ++r) {
                const uint64_t key = open ? order64(worth) : 0;
                const uint32_t h = wave_max((uint32_t)(key >> 32));
                const bool in = (uint32_t)(key >> 32) == h;
                const uint32_t l = wave_max(in ? (uint32_t)key : 0u);
                if (!(h | l)) break;
                const uint64_t who = __ballot(in && (uint32_t)key == l);
                const int winner = __ffsll((unsigned long long)who) - 1;
                kept |= 1ull << winner;
                open = open && lane != winner;
            }
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane * EPL + j, at = e < a.E ? e / size * L : 0;
                if (!((kept >> at) & 1)) {
                    hi[j] = 0;
                    if constexpr (kWide) lo[j] = 0;
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
        // K rounds; lane k keeps choice k
        int chosen = -1;
        float chosen_x = 0.f;
        for (int k = 0; k < a.K; ++k) {
            uint32_t bh = 0, bl = 0;
            int bj = 0;
            float bx = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const bool better = kWide ? (hi[j] > bh || (hi[j] == bh && lo[kWide ? j : 0] > bl)) : hi[j] > bh;
                if (better) {
                    bh = hi[j];
                    if constexpr (kWide) bl = lo[j];
                    bj = j;
                    bx = x[j];
                }
            }
            const uint32_t h = wave_max(bh);
            uint64_t who = __ballot(bh == h);
            if (h == 0) break;                     // nothing left (a live rank's high word is never 0)
            if (kWide && __popcll(who) > 1) {
                const uint32_t l = wave_max(bh == h ? bl : 0u);
                who &= __ballot(bl == l);
            }
            const int winner = __ffsll((unsigned long long)who) - 1;
            const int e = __shfl(lane * EPL + bj, winner);
            const float ex = __shfl(bx, winner);
            if (lane == k) {
                chosen = e;
                chosen_x = ex;
            }
            if (lane == winner) {
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (j == bj) {
                        hi[j] = 0;
                        if constexpr (kWide) lo[j] = 0;
                    }
            }
        }
        // renormalized, softmax's common factor cancels: taken relative to the largest chosen logit, the sum
        // cannot underflow where a bias or the groups left the largest logits out
        if (!kSigmoid && a.renorm) {
            top = wave_max(chosen >= 0 ? chosen_x : -__builtin_inff());
            total = 1.0;
        }
        double s = 0.0;
        if (chosen >= 0)
            s = kSigmoid ? sigmoid64(chosen_x) : exp((double)chosen_x - (double)top) / total;
        if (a.renorm) {
            const double sum = wave_sum(s);
            s = sum > 0.0 ? s / sum : 0.0;
        }
        if (lane < a.K) {
            a.idx[t * a.K + lane] = chosen;
            a.weights[t * a.K + lane] = (float)(s * (double)a.scale);
        }
    }
}

// Gradient.  With G_i the sum of dweights over the places that name expert i, n_i their number, s the scores
// and S the sum of n_i s_i:
//   renormalized   ds_i = scale / S * (G_i - n_i * sum_j(G_j s_j) / S),   else   ds_i = scale * G_i
//   sigmoid        dlogit_i = ds_i s_i (1 - s_i)
//   softmax        dlogit_i = s_i (ds_i - sum_j ds_j s_j); renormalized, that sum is 0
// Only softmax without renormalizing reaches experts that were not named, and only it reads all logits
// (kAll); in the other forms the scores' common factor cancels or does not exist.  One wave per token: lane k
// computes the gradient of the expert that place k names, the row is put together in LDS.
template <int EPL, bool kSigmoid, bool kAll, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void router_backward_kernel(RouterArgs a) {
    __shared__ double rows[WAVES][EPL * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double* row = rows[wave];
    for (int64_t t = (int64_t)blockIdx.x * WAVES + wave; t < a.tokens; t += (int64_t)gridDim.x * WAVES) {
        int64_t id = -1;
        float g = 0.f, xk = -__builtin_inff();
        if (lane < a.K) {
            id = a.idx[t * a.K + lane];
            g = a.dweights[t * a.K + lane];
            if (id < 0 || id >= a.E) id = -1;
            else xk = read_value(a.logits, a.type, (size_t)t * a.E + id);
        }
        const int named = (int)id;
        const bool live = named >= 0 && !is_masked(xk);
        xk = clip_inf(xk);
        float x[kAll ? EPL : 1];
        float top;
        double total = 1.0;
        if constexpr (kAll) {
            read_row<EPL>(a.logits, a.type, t, a.E, lane, x);
            top = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                x[j] = is_masked(x[j]) ? -__builtin_inff() : clip_inf(x[j]);
                top = fmaxf(top, x[j]);
            }
            top = wave_max(top);
            total = 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (x[j] > -__builtin_inff()) total += exp((double)x[j] - (double)top);
            total = wave_sum(total);
        } else {
            top = wave_max(live ? xk : -__builtin_inff());
        }
        double s = 0.0, rest = 0.0;
        if (live) {
            s = kSigmoid ? sigmoid64(xk) : exp((double)xk - (double)top) / total;
            if (kSigmoid) rest = sigmoid64(-(double)xk);      // 1 - s without cancellation
        }
        double G = 0.0;
        int n = 0, before = 0;
        for (int k = 0; k < a.K; ++k) {
            const int e = __shfl(named, k);
            const float gk = __shfl(g, k);
            if (e == named) {
                G += (double)gk;
                ++n;
                before += k < lane;
            }
        }
        const double gs = wave_sum(live ? (double)g * s : 0.0);
        const double S = a.renorm ? wave_sum(s) : 1.0;
        double d = 0.0;
        if (live) {
            if (a.renorm) {
                d = S > 0.0 ? s / S * (G - n * (gs / S)) : 0.0;
                if (kSigmoid) d *= rest;
            } else {
                d = kSigmoid ? G * s * rest : s * (G - gs);
            }
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            double base = 0.0;
            if constexpr (kAll)
                if (x[j] > -__builtin_inff()) base = exp((double)x[j] - (double)top) / total * -gs;
            row[j * 64 + lane] = base;               // expert lane * EPL + j, kept where this lane reads it
        }
        __builtin_amdgcn_wave_barrier();
        if (named >= 0 && before == 0) row[named % EPL * 64 + named / EPL] = d;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane * EPL + j;
            if (e < a.E) write_value(a.dlogits, a.type, (size_t)t * a.E + e, row[j * 64 + lane] * (double)a.scale);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------- ordering
struct OrderArgs {
    const int64_t* idx;
    int32_t *offsets, *order, *slot, *hist;
    int pairs, first, experts, chunks, per_chunk;   // per_chunk pairs per work-group
};

__device__ __forceinline__ int local_of(const OrderArgs& a, int p) {
    const int64_t e = a.idx[p];
    return e >= a.first && e < (int64_t)a.first + a.experts ? (int)(e - a.first) : -1;
}

// Lanes of the wave with the same expert as this one (experts < 4096: 12 bits).
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
    uint64_t m = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e >> b) & 1);
        m &= (e >> b) & 1 ? set : ~set;
    }
    return m;
}

// Rank the pairs lo .. hi-1 by one wave: `next` (LDS) holds the next free place of every expert.
__device__ __forceinline__ void place_pairs(const OrderArgs& a, int lo, int hi, int* next, int lane, int bits) {
    for (int p0 = lo; p0 < hi; p0 += 64) {
        const int p = p0 + lane;
        const int e = p < hi ? local_of(a, p) : -1;
        const uint64_t same = same_expert(e, bits);
        int place = -1;
        if (e >= 0) {
            const int before = __popcll(same & lanemask_lt());
            const int base = next[e];
            place = base + before;
            a.order[place] = p;
        }
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && (same & lanemask_lt()) == 0) next[e] = place + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (p < hi) a.slot[p] = place;
    }
}

__device__ __forceinline__ int bits_of(int experts) { return experts > 1 ? 32 - __clz(experts - 1) : 0; }

// Few pairs: everything in one work-group of 16 waves.  Dynamic LDS: int [16][experts], then int [17].
__global__ __launch_bounds__(1024) void order_small_kernel(OrderArgs a) {
    extern __shared__ int lds[];
    int* sums = lds + 16 * a.experts;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < 16 * a.experts; i += 1024) lds[i] = 0;
    __syncthreads();
    const int per = ((a.pairs + 15) / 16 + 63) / 64 * 64;
    const int lo = min(wave * per, a.pairs), hi = min(lo + per, a.pairs);
    for (int p = lo + lane; p < hi; p += 64) {
        const int e = local_of(a, p);
        if (e >= 0) atomicAdd(&lds[wave * a.experts + e], 1);
    }
    __syncthreads();
    // thread e: the expert's total (experts <= 512), then an exclusive prefix over the experts
    int count = 0;
    if (tid < a.experts)
        for (int w = 0; w < 16; ++w) count += lds[w * a.experts + tid];
    int incl = wave_prefix(count, lane);
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    if (wave == 0) {
        const int v = lane < 16 ? sums[lane] : 0;
        const int s = wave_prefix(v, lane);
        if (lane < 16) sums[lane] = s - v;
        if (lane == 15) sums[16] = s;
    }
    __syncthreads();
    if (tid < a.experts) {
        int at = sums[wave] + incl - count;
        a.offsets[tid] = at;
        for (int w = 0; w < 16; ++w) {
            const int c = lds[w * a.experts + tid];
            lds[w * a.experts + tid] = at;
            at += c;
        }
    }
    const int all = sums[16];
    if (tid == 0) a.offsets[a.experts] = all;
    __syncthreads();
    place_pairs(a, lo, hi, lds + wave * a.experts, lane, bits_of(a.experts));
    for (int i = all + tid; i < a.pairs; i += 1024) a.order[i] = -1;
}

// Many pairs, three launches.  1: every chunk's counts, hist[chunk][expert].
__global__ __launch_bounds__(256) void order_count_kernel(OrderArgs a) {
    extern __shared__ int lds[];
    for (int i = threadIdx.x; i < a.experts; i += 256) lds[i] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.per_chunk, hi = min(lo + a.per_chunk, (int64_t)a.pairs);
    for (int64_t p = lo + threadIdx.x; p < hi; p += 256) {
        const int e = local_of(a, (int)p);
        if (e >= 0) atomicAdd(&lds[e], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.experts; i += 256) a.hist[(size_t)blockIdx.x * a.experts + i] = lds[i];
}

// 2: hist becomes every chunk's first place within its expert, offsets the experts' first places.  One
// work-group; thread i handles experts i, i + 1024, ...
__global__ __launch_bounds__(1024) void order_scan_kernel(OrderArgs a) {
    __shared__ int sums[17];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int base = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 1024) {
        const int e = e0 + tid;
        int count = 0;
        if (e < a.experts)
            for (int c = 0; c < a.chunks; ++c) {
                const size_t i = (size_t)c * a.experts + e;
                const int v = a.hist[i];
                a.hist[i] = count;
                count += v;
            }
        const int incl = wave_prefix(count, lane);
        if (lane == 63) sums[wave] = incl;
        __syncthreads();
        if (wave == 0) {
            const int v = lane < 16 ? sums[lane] : 0;
            const int s = wave_prefix(v, lane);
            if (lane < 16) sums[lane] = s - v;
            if (lane == 15) sums[16] = s;
        }
        __syncthreads();
        if (e < a.experts) a.offsets[e] = base + sums[wave] + incl - count;
        base += sums[16];
        __syncthreads();
    }
    if (tid == 0) a.offsets[a.experts] = base;
}

// 3: places.  Dynamic LDS: int [4][experts].
__global__ __launch_bounds__(256) void order_place_kernel(OrderArgs a) {
    extern __shared__ int lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t first = (int64_t)blockIdx.x * a.per_chunk;
    const int per = a.per_chunk / 4;
    const int64_t end = min(first + a.per_chunk, (int64_t)a.pairs);
    const int lo = (int)min(first + (int64_t)wave * per, end), hi = (int)min((int64_t)lo + per, end);
    for (int i = tid; i < 4 * a.experts; i += 256) lds[i] = 0;
    __syncthreads();
    for (int p = lo + lane; p < hi; p += 64) {
        const int e = local_of(a, p);
        if (e >= 0) atomicAdd(&lds[wave * a.experts + e], 1);
    }
    __syncthreads();
    for (int e = tid; e < a.experts; e += 256) {
        int at = a.offsets[e] + a.hist[(size_t)blockIdx.x * a.experts + e];
        for (int w = 0; w < 4; ++w) {
            const int c = lds[w * a.experts + e];
            lds[w * a.experts + e] = at;
            at += c;
        }
    }
    __syncthreads();
    place_pairs(a, lo, hi, lds + wave * a.experts, lane, bits_of(a.experts));
    for (int64_t i = max(first, (int64_t)a.offsets[a.experts]) + tid; i < end; i += 256) a.order[i] = -1;
}

// Pairs per work-group of the three-launch form: a multiple of 4 waves x 64, and at most 1024 chunks for the scan.
int chunk_pairs(int64_t pairs) {
    const int64_t least = 4 * kPairsPerWave, by_chunks = (pairs + 1023) / 1024;
    return (int)((by_chunks < least ? least : by_chunks) + 255) / 256 * 256;
}

int32_t check_router(const mega_moe_router_config* c) {
    if (!c || c->tokens < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (c->num_experts < 1 || c->num_experts > MEGA_MOE_MAX_EXPERTS || c->topk < 1 || c->topk > MEGA_MOE_MAX_TOPK ||
        c->topk > c->num_experts || c->tokens >= (int64_t)1 << 31 || c->tokens * c->topk >= (int64_t)1 << 31 ||
        (c->score != MEGA_MOE_SCORE_SOFTMAX && c->score != MEGA_MOE_SCORE_SIGMOID) || c->num_groups < 1 ||
        c->num_groups > 64 || c->num_experts % c->num_groups || c->topk_groups < 1 ||
        c->topk_groups > c->num_groups || (c->group_top != 1 && c->group_top != 2) ||
        c->dtype < MEGA_MOE_BF16 || c->dtype > MEGA_MOE_FP32 || !(c->scale - c->scale == 0.0f))
        return MEGA_MOE_ERR_UNSUPPORTED;
    return MEGA_MOE_OK;
}

RouterArgs args_of(const mega_moe_router_config* c) {
    RouterArgs a{};
    a.tokens = c->tokens;
    a.E = c->num_experts;
    a.K = c->topk;
    a.G = c->num_groups;
    a.kept = c->topk_groups;
    a.gtop = c->group_top;
    a.scale = c->scale;
    a.renorm = c->renormalize != 0;
    a.type = c->dtype;
    return a;
}

uint32_t router_grid(int64_t tokens, int waves) {
    const int64_t g = (tokens + waves - 1) / waves;
    return (uint32_t)(g < (1 << 20) ? g : 1 << 20);
}

template <int EPL, bool kSigmoid, bool kWide, bool kGroups>
hipError_t launch_router(const RouterArgs& a, hipStream_t st) {
    // the groups' values take EPL * 512 bytes of LDS per wave
    constexpr int WAVES = kGroups && EPL > 16 ? 1 : 4;
    hipLaunchKernelGGL((router_kernel<EPL, kSigmoid, kWide, kGroups, WAVES>), dim3(router_grid(a.tokens, WAVES)),
                       dim3(WAVES * 64), 0, st, a);
    return hipGetLastError();
}
template <int EPL>
hipError_t pick_router(const RouterArgs& a, bool sigmoid, hipStream_t st) {
    switch ((sigmoid ? 4 : 0) | (a.bias ? 2 : 0) | (a.G > 1 ? 1 : 0)) {
        case 0: return launch_router<EPL, false, false, false>(a, st);
        case 1: return launch_router<EPL, false, false, true>(a, st);
        case 2: return launch_router<EPL, false, true, false>(a, st);
        case 3: return launch_router<EPL, false, true, true>(a, st);
        case 4: return launch_router<EPL, true, false, false>(a, st);
        case 5: return launch_router<EPL, true, false, true>(a, st);
        case 6: return launch_router<EPL, true, true, false>(a, st);
        default: return launch_router<EPL, true, true, true>(a, st);
    }
}
template <int EPL>
hipError_t pick_backward(const RouterArgs& a, bool sigmoid, hipStream_t st) {
    constexpr int WAVES = EPL > 16 ? 1 : 4;
    const dim3 grid(router_grid(a.tokens, WAVES)), block(WAVES * 64);
    if (sigmoid) hipLaunchKernelGGL((router_backward_kernel<EPL, true, false, WAVES>), grid, block, 0, st, a);
    else if (a.renorm) hipLaunchKernelGGL((router_backward_kernel<EPL, false, false, WAVES>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((router_backward_kernel<EPL, false, true, WAVES>), grid, block, 0, st, a);
    return hipGetLastError();
}

bool aligned16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int32_t mega_moe_router_topk(const mega_moe_router_config* cfg, const void* logits, const float* bias,
                             int64_t* topk_idx, float* topk_weights, void* stream) {
    const int32_t rc = check_router(cfg);
    if (rc) return rc;
    if (bias && !aligned16(bias)) return MEGA_MOE_ERR_INVALID_ARG;
    if (cfg->tokens == 0) return MEGA_MOE_OK;
    if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(topk_weights)) return MEGA_MOE_ERR_INVALID_ARG;
    RouterArgs a = args_of(cfg);
    a.logits = logits;
    a.bias = bias;
    a.idx = topk_idx;
    a.weights = topk_weights;
    const bool sigmoid = cfg->score == MEGA_MOE_SCORE_SIGMOID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = a.E <= 64     ? pick_router<1>(a, sigmoid, st)
                         : a.E <= 128  ? pick_router<2>(a, sigmoid, st)
                         : a.E <= 256  ? pick_router<4>(a, sigmoid, st)
                         : a.E <= 512  ? pick_router<8>(a, sigmoid, st)
                         : a.E <= 1024 ? pick_router<16>(a, sigmoid, st)
                                       : pick_router<64>(a, sigmoid, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_router_backward(const mega_moe_router_config* cfg, const float* dweights, const void* logits,
                                 const int64_t* topk_idx, void* dlogits, void* stream) {
    const int32_t rc = check_router(cfg);
    if (rc) return rc;
    if (cfg->tokens == 0) return MEGA_MOE_OK;
    if (!aligned16(dweights) || !aligned16(logits) || !aligned16(topk_idx) || !aligned16(dlogits))
        return MEGA_MOE_ERR_INVALID_ARG;
    RouterArgs a = args_of(cfg);
    a.logits = logits;
    a.dweights = dweights;
    a.idx = const_cast<int64_t*>(topk_idx);
    a.dlogits = dlogits;
    const bool sigmoid = cfg->score == MEGA_MOE_SCORE_SIGMOID;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = a.E <= 64     ? pick_backward<1>(a, sigmoid, st)
                         : a.E <= 128  ? pick_backward<2>(a, sigmoid, st)
                         : a.E <= 256  ? pick_backward<4>(a, sigmoid, st)
                         : a.E <= 512  ? pick_backward<8>(a, sigmoid, st)
                         : a.E <= 1024 ? pick_backward<16>(a, sigmoid, st)
                                       : pick_backward<64>(a, sigmoid, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_group_workspace_bytes(int64_t pairs, int32_t num_local_experts, uint64_t* bytes_out) {
    if (!bytes_out || pairs < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (pairs >= (int64_t)1 << 31 || num_local_experts < 1 || num_local_experts > MEGA_MOE_MAX_EXPERTS)
        return MEGA_MOE_ERR_UNSUPPORTED;
    const int64_t per = chunk_pairs(pairs);
    *bytes_out = (uint64_t)((pairs + per - 1) / per + 1) * num_local_experts * 4;
    return MEGA_MOE_OK;
}

int32_t mega_moe_group_by_expert(const int64_t* topk_idx, int64_t pairs, int32_t first_expert,
                                 int32_t num_local_experts, int32_t* offsets, int32_t* order, int32_t* slot,
                                 void* workspace, uint64_t workspace_bytes, void* stream) {
    uint64_t need = 0;
    const int32_t rc = mega_moe_group_workspace_bytes(pairs, num_local_experts, &need);
    if (rc) return rc;
    if (first_expert < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!aligned16(offsets) || !aligned16(workspace) ||
        (pairs > 0 && (!aligned16(topk_idx) || !aligned16(order) || !aligned16(slot))))
        return MEGA_MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    hipStream_t st = static_cast<hipStream_t>(stream);
    OrderArgs a{topk_idx, offsets, order, slot, static_cast<int32_t*>(workspace), (int)pairs, first_expert,
                num_local_experts, 0, 0};
    if (pairs <= kOneGroupPairs && num_local_experts <= kOneGroupExperts) {
        hipLaunchKernelGGL(order_small_kernel, dim3(1), dim3(1024), (16 * num_local_experts + 17) * sizeof(int), st, a);
        return hipGetLastError() == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
    }
    a.per_chunk = chunk_pairs(pairs);
    a.chunks = (int)((pairs + a.per_chunk - 1) / a.per_chunk);
    const dim3 chunks(a.chunks > 0 ? a.chunks : 1), block(256);
    hipLaunchKernelGGL(order_count_kernel, chunks, block, num_local_experts * sizeof(int), st, a);
    hipLaunchKernelGGL(order_scan_kernel, dim3(1), dim3(1024), 0, st, a);
    hipLaunchKernelGGL(order_place_kernel, chunks, block, 4 * num_local_experts * sizeof(int), st, a);
    return hipGetLastError() == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
