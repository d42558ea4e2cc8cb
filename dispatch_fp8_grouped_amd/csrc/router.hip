// The router around the fused layer (include/mega_moe_ops.h): the choice and weights of each token's experts,
// the gradient of the weights, and the ordering of the chosen pairs by expert.
//
// Choice: LANES lanes per token (a wave, or a quarter of one); lane l of them holds experts l*EPL .. l*EPL + EPL-1
// (so the lowest lane of a tie holds the lowest expert).  Without a bias the logit and the expert's number make one
// key, all different: each lane sorts its own once, and a round is a maximum over the lanes' first ones.  With a bias
// the fp64 score + bias is the rank, as two unsigned words: a round takes the largest high word, and only where
// several lanes share it do the low words decide.  What bounds it is instruction issue, and the rounds cost the same
// whether a wave serves one token or four, so many tokens take a quarter wave each.  32768 tokens x 256 experts,
// top 8, bf16: 38 us with a wave each and fp64 keys, 16 with a quarter, 11.5 with 32-bit keys, both loads in flight
// and the chosen logits taken from the keys (the bytes: 5).  Few tokens take a whole wave, whose lanes have fewer
// experts to walk (1024 x 256, fp32, sigmoid with bias and groups: 8 us).
//
// Scores are computed in fp64 (exp of the C library's device functions): two scores that differ in fp32
// logits then differ in rank, and the choice does not hang on a rounding of exp.
#include <type_traits>

#include "gemm_tiles.h"

namespace mm {
namespace {

constexpr int kPairsPerWave = 256;           // least pairs that one wave of the ordering places, 64 at a time
constexpr int kFewPairs = 32768;             // up to here one launch orders everything
constexpr int kFewExperts = 512;             // 36 KB of counters

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
// This lane's EPL values v(j) of a row of E, wide where read_lane reads wide.
template <int EPL, class V, class F>
__device__ __forceinline__ void write_lane(V* row, int E, int lane, F value) {
    constexpr int kWide = EPL * (int)sizeof(V) < 16 ? EPL : 16 / (int)sizeof(V);
    struct __align__(kWide * sizeof(V)) Wide { V v[kWide]; };
    const int e0 = lane * EPL;
    if (E % EPL == 0) {
        if (e0 >= E) return;
#pragma unroll
        for (int j = 0; j < EPL; j += kWide) {
            Wide w;
#pragma unroll
            for (int i = 0; i < kWide; ++i) w.v[i] = value(j + i);
            *reinterpret_cast<Wide*>(row + e0 + j) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (e0 + j < E) row[e0 + j] = value(j);
    }
}
template <int EPL, class F>
__device__ __forceinline__ void write_row(void* p, int type, int64_t t, int E, int lane, F v) {
    const size_t at = (size_t)t * E;
    if (type == MEGA_MOE_FP32)
        write_lane<EPL>(static_cast<float*>(p) + at, E, lane, [&](int j) { return (float)v(j); });
    else if (type == MEGA_MOE_BF16)
        write_lane<EPL>(static_cast<uint16_t*>(p) + at, E, lane, [&](int j) { return (uint16_t)Bf16::pack((float)v(j), 0.f); });
    else
        write_lane<EPL>(static_cast<_Float16*>(p) + at, E, lane, [&](int j) { return (_Float16)(float)v(j); });
}

// This lane's EPL logits of a row of E; -inf past the row.  Where E is a multiple of EPL, every lane's
// values lie in the row or all behind it, and are aligned to their own size: one or a few wide loads.
template <int EPL, class V, class F>
__device__ __forceinline__ void read_lane(const V* row, int E, int lane, float (&x)[EPL], F value) {
    constexpr int kWide = EPL * (int)sizeof(V) < 16 ? EPL : 16 / (int)sizeof(V);
    struct __align__(kWide * sizeof(V)) Wide { V v[kWide]; };
    const int e0 = lane * EPL;
    if (E % EPL == 0) {
        // lanes behind the row read its last values, and drop them: no branch between the loads
        const Wide* from = reinterpret_cast<const Wide*>(row + min(e0, E - EPL));
        Wide w[EPL / kWide];
#pragma unroll
        for (int j = 0; j < EPL / kWide; ++j) w[j] = from[j];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float v = value(w[j / kWide].v[j % kWide]);
            x[j] = e0 < E ? v : -__builtin_inff();
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

// A logit and its expert as one number, so that of equal logits the lower expert's number is larger; all are
// different, and above kNone unless the logit is masked.  fp32: an fp64 number, of whose 53 bits the logit takes 24
// and the expert the low 12.  bf16 and fp16: their values as fp32 end with 12 zeros at least, which the expert takes;
// unsigned integers in the order of the numbers cost half the registers and less than half the instructions.
constexpr int kExpertMask = MEGA_MOE_MAX_EXPERTS - 1;
static_assert(MEGA_MOE_MAX_EXPERTS == 1 << 12, "12 bits");
template <class Key>
struct Ranked;
template <>
struct Ranked<double> {
    static constexpr double kNone = -__builtin_inff();
    static __device__ __forceinline__ double of(float x, int e) {
        const uint64_t u = (uint64_t)__double_as_longlong((double)(clip_inf(x) + 0.0f));        // -0 ranks with +0
        const double key = __longlong_as_double((long long)(u | (uint64_t)(u >> 63 ? e : kExpertMask - e)));
        return is_masked(x) ? kNone : key;
    }
    static __device__ __forceinline__ int expert(double key) {
        const uint64_t u = (uint64_t)__double_as_longlong(key);
        const int low = (int)(u & kExpertMask);
        return u >> 63 ? low : kExpertMask - low;
    }
    static __device__ __forceinline__ float logit(double key) {
        return (float)__longlong_as_double(__double_as_longlong(key) & ~(long long)kExpertMask);
    }
};
template <>
struct Ranked<uint32_t> {
    static constexpr uint32_t kNone = 0x007FFFFFu;                 // -inf with any expert is not above it
    static __device__ __forceinline__ uint32_t of(float x, int e) {
        const uint32_t u = __float_as_uint(fmaxf(x, -__builtin_inff()) + 0.0f);                 // NaN becomes -inf
        return ((u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) & ~(uint32_t)kExpertMask) + (uint32_t)(kExpertMask - e);
    }
    static __device__ __forceinline__ int expert(uint32_t key) { return kExpertMask - (int)(key & kExpertMask); }
    static __device__ __forceinline__ float logit(uint32_t key) {
        return __uint_as_float((key >> 31 ? key ^ 0x80000000u : ~key) & ~(uint32_t)kExpertMask);
    }
};
template <>
struct Ranked<uint64_t> {
    static constexpr uint64_t kNone = 0;
};

__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) { return min(a, b); }

// Sort n numbers, the largest first (Batcher's odd-even merge network; n a power of two)
template <int n, class Key>
__device__ __forceinline__ void sort_down(Key (&v)[n]) {
#pragma unroll
    for (int p = 1; p < n; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < n; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < n && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const Key a = v[i + j], b = v[i + j + k];
                        v[i + j] = larger(a, b);
                        v[i + j + k] = smaller(a, b);
                    }
}

// Unsigned integers in the order of the numbers (no NaN); no number maps to 0.
__device__ __forceinline__ uint64_t order64(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// v of a lane in the other half of 2 d lanes, for a v that is the same in every run of d lanes (DPP quad
// permutations and mirrors; the row and half-wave swaps return both halves)
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xF, 0xF, true);
}
template <int d>
__device__ __forceinline__ uint32_t mirror(uint32_t v) {
    static_assert(d == 1 || d == 2 || d == 4 || d == 8, "within a row of 16 lanes");
    return d == 1 ? dpp<0xB1>(v) : d == 2 ? dpp<0x4E>(v) : d == 4 ? dpp<0x141>(v) : dpp<0x140>(v);
}
__device__ __forceinline__ uint32_t low_word(double v) { return (uint32_t)__double_as_longlong(v); }
__device__ __forceinline__ uint32_t high_word(double v) { return (uint32_t)((uint64_t)__double_as_longlong(v) >> 32); }
__device__ __forceinline__ double from_words(uint32_t lo, uint32_t hi) {
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
template <int d>
__device__ __forceinline__ double mirror(double v) { return from_words(mirror<d>(low_word(v)), mirror<d>(high_word(v))); }

// op over LANES neighbouring lanes (16 or 64), the result in all of them; op's order is fixed by the lane numbers
template <int LANES, class F>
__device__ __forceinline__ uint32_t all_of(uint32_t v, F op) {
    v = op(v, mirror<1>(v));
    v = op(v, mirror<2>(v));
    v = op(v, mirror<4>(v));
    v = op(v, mirror<8>(v));
    if constexpr (LANES == 64) {
        const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(a[0], a[1]);
        const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(b[0], b[1]);
    }
    return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
    return all_of<LANES>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LANES>
__device__ __forceinline__ float max_of(float v) {
    return __uint_as_float(all_of<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
template <int LANES>
__device__ __forceinline__ double max_of(double v) {
    v = fmax(v, mirror<1>(v));
    v = fmax(v, mirror<2>(v));
    v = fmax(v, mirror<4>(v));
    v = fmax(v, mirror<8>(v));
    if constexpr (LANES == 64) {
        auto l = __builtin_amdgcn_permlane16_swap(low_word(v), low_word(v), false, false);
        auto h = __builtin_amdgcn_permlane16_swap(high_word(v), high_word(v), false, false);
        v = fmax(from_words(l[0], h[0]), from_words(l[1], h[1]));
        l = __builtin_amdgcn_permlane32_swap(low_word(v), low_word(v), false, false);
        h = __builtin_amdgcn_permlane32_swap(high_word(v), high_word(v), false, false);
        v = fmax(from_words(l[0], h[0]), from_words(l[1], h[1]));
    }
    return v;
}
// Sums of fp64 (the two operands of an addition swap between lanes, which changes nothing)
template <int LANES>
__device__ __forceinline__ double sum_of(double v) {
    v += mirror<1>(v);
    v += mirror<2>(v);
    v += mirror<4>(v);
    v += mirror<8>(v);
    if constexpr (LANES == 64) {
        auto l = __builtin_amdgcn_permlane16_swap(low_word(v), low_word(v), false, false);
        auto h = __builtin_amdgcn_permlane16_swap(high_word(v), high_word(v), false, false);
        v = from_words(l[0], h[0]) + from_words(l[1], h[1]);
        l = __builtin_amdgcn_permlane32_swap(low_word(v), low_word(v), false, false);
        h = __builtin_amdgcn_permlane32_swap(high_word(v), high_word(v), false, false);
        v = from_words(l[0], h[0]) + from_words(l[1], h[1]);
    }
    return v;
}
// Lanes of this token for which `p` holds, as bits from 0
template <int LANES>
__device__ __forceinline__ uint64_t lanes_with(bool p) {
    const uint64_t all = __ballot(p);
    return LANES == 64 ? all : (all >> (__lane_id() & ~(LANES - 1))) & ((1ull << (LANES & 63)) - 1);
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// A pair of largest values, merged
__device__ __forceinline__ void merge_top2(double& a, double& b, double c, double d) {
    const double hi = fmax(a, c), lo = fmin(a, c);
    b = fmax(lo, fmax(b, d));
    a = hi;
}

// Key: a logit with its expert as double or uint32_t (with_expert), or uint64_t for ranks as two words without
// the expert (with a bias, or with too many experts to a lane to sort).  A work-group's tokens follow each other.
template <int EPL, int LANES, bool kSigmoid, class Key, bool kGroups, int WAVES>
__global__ __launch_bounds__(WAVES * 64, (EPL <= 16 && !std::is_same<Key, uint64_t>::value && !kGroups ? 4 : 1)) void
router_kernel(RouterArgs a) {
    constexpr bool kWide = std::is_same<Key, uint64_t>::value;
    constexpr int kTokens = WAVES * 64 / LANES;
    __shared__ double values[kGroups ? kTokens : 1][kGroups ? EPL * LANES : 1];
    const int lane = threadIdx.x % LANES, mine = threadIdx.x / LANES, wave = threadIdx.x >> 6;
    const double none = -__builtin_inf();
    // a wave whose last tokens do not exist repeats the last one for them, and does not store
    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 + wave * (64 / LANES) < a.tokens; t0 += (int64_t)gridDim.x * kTokens) {
        const bool real = t0 + mine < a.tokens;
        const int64_t t = real ? t0 + mine : a.tokens - 1;
        float x[EPL];
        bool live[EPL];
        float top = -__builtin_inff();
        read_row<EPL>(a.logits, a.type, t, a.E, lane, x);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            live[j] = !is_masked(x[j]);
            if constexpr (kWide) x[j] = clip_inf(x[j]);
        }
        // softmax needs its largest logit and its sum where the scores themselves enter the result; where they
        // are divided by the chosen ones' sum both cancel
        const bool by_score = (kWide && a.bias) || (kGroups && a.gtop == 2);
        double total = 1.0;
        if (!kSigmoid && (by_score || !a.renorm)) {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (live[j]) top = fmaxf(top, clip_inf(x[j]));
            top = max_of<LANES>(top);              // -inf where everything is masked
            total = 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (live[j]) total += exp((double)clip_inf(x[j]) - (double)top);
            total = sum_of<LANES>(total);
        }
        uint32_t hi[kWide ? EPL : 1], lo[kWide ? EPL : 1];
        Key key[kWide ? 1 : EPL];
        constexpr Key none_key = Ranked<Key>::kNone;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane * EPL + j;
            // clipped as in the expert's key: a group of +inf ties with one of the largest number
            double rank = x[j], worth = kWide ? x[j] : clip_inf(x[j]);
            if (by_score && live[j]) {
                const double s = kSigmoid ? sigmoid64(x[j]) : exp((double)clip_inf(x[j]) - (double)top) / total;
                worth = s;
                if (kWide && a.bias) {
                    worth = rank = s + (double)a.bias[e];
                    live[j] = rank > none;         // not -inf, not NaN
                }
            }
            if constexpr (kWide) {
                const uint64_t word = live[j] ? order64(rank) : 0;
                hi[j] = (uint32_t)(word >> 32);
                lo[j] = (uint32_t)word;
            } else {
                key[j] = Ranked<Key>::of(x[j], e);
            }
            if constexpr (kGroups) values[mine][e] = live[j] ? worth : none;
        }
        if constexpr (kGroups) {
            // L lanes per group (a power of two); group g's lanes are g*L .. g*L + L-1
            int L = 1;
            while (L * 2 * a.G <= LANES) L *= 2;
            const int size = a.E / a.G, g = lane / L;
            double first = none, second = none;
            __builtin_amdgcn_wave_barrier();
            if (g < a.G)
                for (int i = lane % L; i < size; i += L) merge_top2(first, second, values[mine][g * size + i], none);
            auto meet = [&](auto other) {
                const double c = other(first), d = other(second);
                merge_top2(first, second, c, d);
            };
            if (L > 1) meet([](double v) { return mirror<1>(v); });
            if (L > 2) meet([](double v) { return mirror<2>(v); });
            if (L > 4) meet([](double v) { return mirror<4>(v); });
            if (L > 8) meet([](double v) { return mirror<8>(v); });
            if (L > 16) meet([](double v) { return __shfl_xor(v, 16); });
            // a group's worth: its best, or the sum of its two best where it has two
            double worth = first;
            if (a.gtop == 2 && second > none) worth += second;
            bool open = (lane % L) == 0 && g < a.G && first > none;
            uint64_t kept = 0;                     // bit of every kept group's first lane
            for (int r = 0; r < a.kept; ++r) {
                const double best = max_of<LANES>(open ? worth : none);
                const uint64_t who = lanes_with<LANES>(open && worth == best);
                if (who) {
                    const int winner = __ffsll((unsigned long long)who) - 1;
                    kept |= 1ull << winner;
                    open = open && lane != winner;
                }
            }
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane * EPL + j, at = e < a.E ? e / size * L : 0;
                if (!((kept >> at) & 1)) {
                    if constexpr (kWide) hi[j] = lo[j] = 0;
                    else key[j] = none_key;
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
        // K rounds; lane k keeps choice k
        int chosen = -1;
        float chosen_x = -__builtin_inff();
        if constexpr (kWide) {
            // a live rank's high word is never 0
            for (int k = 0; k < a.K; ++k) {
                uint32_t bh = 0, bl = 0;
                int bj = 0;
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (hi[j] > bh || (hi[j] == bh && lo[j] > bl)) {
                        bh = hi[j];
                        bl = lo[j];
                        bj = j;
                    }
                const uint32_t h = max_of<LANES>(bh);
                uint64_t who = lanes_with<LANES>(bh == h);
                if (__any(__popcll(who) > 1)) {
                    const uint32_t l = max_of<LANES>(bh == h ? bl : 0u);
                    who = lanes_with<LANES>(bh == h && bl == l);
                }
                const int winner = h ? __ffsll((unsigned long long)who) - 1 : -1;
                const int e = __shfl(lane * EPL + bj, (threadIdx.x & 63 & ~(LANES - 1)) + max(winner, 0));
                if (lane == k && winner >= 0) chosen = e;
                const int gone = lane == winner ? bj : -1;
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (j == gone) hi[j] = lo[j] = 0;
            }
        } else {
            // every lane's experts sorted once: a round looks at the lanes' first ones, and the lane that had the
            // largest moves up.  Only the first K of a lane can be reached.
            sort_down(key);
            Key mine_key = none_key;
            auto rounds = [&](auto depth) {
                constexpr int kDepth = decltype(depth)::value;
                for (int k = 0; k < a.K; ++k) {
                    const Key best = max_of<LANES>(key[0]);
                    if (lane == k) mine_key = best;
                    const bool mine_won = key[0] == best;
#pragma unroll
                    for (int j = 0; j < kDepth; ++j) {
                        const Key next = j + 1 < EPL ? key[j + 1 < EPL ? j + 1 : 0] : none_key, now = key[j];
                        key[j] = mine_won ? next : now;
                    }
                }
            };
            if (EPL > 8 && a.K <= 8) rounds(std::integral_constant<int, EPL < 8 ? EPL : 8>{});
            else rounds(std::integral_constant<int, EPL>{});
            if (mine_key > none_key) {
                chosen = Ranked<Key>::expert(mine_key);
                chosen_x = clip_inf(Ranked<Key>::logit(mine_key));
            }
        }
        if (kWide && chosen >= 0) chosen_x = clip_inf(read_value(a.logits, a.type, (size_t)t * a.E + chosen));   // from the cache
        // renormalized, softmax's common factor cancels: taken relative to the largest chosen logit, the sum
        // cannot underflow where a bias or the groups left the largest logits out
        if (!kSigmoid && a.renorm) {
            top = max_of<LANES>(chosen_x);
            total = 1.0;
        }
        double s = 0.0;
        if (chosen >= 0)
            s = kSigmoid ? sigmoid64(chosen_x) : exp((double)chosen_x - (double)top) / total;
        if (a.renorm) {
            const double sum = sum_of<LANES>(s);
            s = sum > 0.0 ? s / sum : 0.0;
        }
        if (real && lane < a.K) {
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
// (kAll); in the other forms the scores' common factor cancels or does not exist.  LANES lanes per token as in the
// choice: lane k computes the gradient of the expert that place k names, the row is put together in LDS.
template <int EPL, int LANES, bool kSigmoid, bool kAll, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void router_backward_kernel(RouterArgs a) {
    constexpr int kTokens = WAVES * 64 / LANES;
    __shared__ double rows[kTokens][EPL * LANES];
    const int lane = threadIdx.x % LANES, mine = threadIdx.x / LANES, wave = threadIdx.x >> 6;
    const int lane0 = threadIdx.x & 63 & ~(LANES - 1);
    double* row = rows[mine];
    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 + wave * (64 / LANES) < a.tokens; t0 += (int64_t)gridDim.x * kTokens) {
        const bool real = t0 + mine < a.tokens;
        const int64_t t = real ? t0 + mine : a.tokens - 1;
        float x[kAll ? EPL : 1];
        if constexpr (kAll) read_row<EPL>(a.logits, a.type, t, a.E, lane, x);
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
        double base[kAll ? EPL : 1];               // scores of this lane's experts
        float top;
        double total = 1.0;
        if constexpr (kAll) {
            top = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                x[j] = is_masked(x[j]) ? -__builtin_inff() : clip_inf(x[j]);
                top = fmaxf(top, x[j]);
            }
            top = max_of<LANES>(top);
            total = 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                base[j] = x[j] > -__builtin_inff() ? exp((double)x[j] - (double)top) : 0.0;
                total += base[j];
            }
            total = sum_of<LANES>(total);
        } else {
            top = max_of<LANES>(live ? xk : -__builtin_inff());
        }
        double s = 0.0, rest = 0.0;
        if (live) {
            s = kSigmoid ? sigmoid64(xk) : exp((double)xk - (double)top) / total;
            if (kSigmoid) rest = sigmoid64(-(double)xk);      // 1 - s without cancellation
        }
        double G = 0.0;
        int n = 0, before = 0;
        for (int k = 0; k < a.K; ++k) {
            const int e = __shfl(named, lane0 + k);
            const float gk = __shfl(g, lane0 + k);
            if (e == named) {
                G += (double)gk;
                ++n;
                before += k < lane;
            }
        }
        const double gs = sum_of<LANES>(live ? (double)g * s : 0.0);
        const double S = a.renorm ? sum_of<LANES>(s) : 1.0;
        double d = 0.0;
        if (live) {
            if (a.renorm) {
                d = S > 0.0 ? s / S * (G - n * (gs / S)) : 0.0;
                if (kSigmoid) d *= rest;
            } else {
                d = kSigmoid ? G * s * rest : s * (G - gs);
            }
        }
        const double down = total > 0.0 ? -gs / total : 0.0;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            // expert lane * EPL + j, kept where this lane reads it; a masked expert's score is 0, whatever gs
            row[j * LANES + lane] = kAll && base[kAll ? j : 0] > 0.0 ? base[kAll ? j : 0] * down : 0.0;
        __builtin_amdgcn_wave_barrier();
        if (named >= 0 && before == 0) row[named % EPL * LANES + named / EPL] = d;
        __builtin_amdgcn_wave_barrier();
        if (real) write_row<EPL>(a.dlogits, a.type, t, a.E, lane, [&](int j) { return row[j * LANES + lane] * (double)a.scale; });
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------- ordering
struct OrderArgs {
    const int64_t* idx;
    int32_t *offsets, *order, *slot;
    int32_t* hist;      // [experts][chunks], then [experts] totals
    int pairs, first, experts, chunks, per_chunk;   // per_chunk pairs per work-group
};

__device__ __forceinline__ int local_id(const OrderArgs& a, int64_t e) {
    return e >= a.first && e < (int64_t)a.first + a.experts ? (int)(e - a.first) : -1;
}
__device__ __forceinline__ int local_of(const OrderArgs& a, int p) { return local_id(a, a.idx[p]); }

// Lanes of the wave with the same expert as this one (experts < 4096: 12 bits).
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
    const uint64_t live = __ballot(e >= 0);
    uint32_t lo = (uint32_t)live, hi = (uint32_t)(live >> 32);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e >> b) & 1);
        const uint32_t other = ((uint32_t)e >> b & 1) - 1;          // all ones where this lane's bit is 0
        lo &= (uint32_t)set ^ other;
        hi &= (uint32_t)(set >> 32) ^ other;
    }
    return (uint64_t)hi << 32 | lo;
}

// Places of 64 consecutive pairs, one wave: lane's pair p goes to expert e (-1: none); `next` (LDS, the wave's
// own) holds the next free place of every expert.
__device__ __forceinline__ void place_pairs(const OrderArgs& a, int e, int p, int hi, int* next, int bits) {
    const uint64_t same = same_expert(e, bits);
    int place = -1;
    if (e >= 0) {
        place = next[e] + __popcll(same & lanemask_lt());
        a.order[place] = p;
    }
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && (same & lanemask_lt()) == 0) next[e] = place + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (p < hi) a.slot[p] = place;
}

__device__ __forceinline__ int bits_of(int experts) { return experts > 1 ? 32 - __clz(experts - 1) : 0; }

// Few pairs, one launch: every work-group counts all pairs and places 1024 of them, 64 to a wave, so that nothing
// passes between work-groups (8192 pairs, 256 experts: 6.0 us; one work-group placing all of them 11, the three
// launches below 10; at 32768 pairs 10.2 against 10.5).  Dynamic LDS: int [16][experts] its own waves' counts, [experts] of the pairs before its
// own, [experts] of those behind, [32].
__global__ __launch_bounds__(1024) void order_few_kernel(OrderArgs a) {
    extern __shared__ int lds[];
    int *before = lds + 16 * a.experts, *behind = before + a.experts, *sums = behind + a.experts;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, own = blockIdx.x, p = own * 1024 + tid;
    for (int i = tid; i < 18 * a.experts; i += 1024) lds[i] = 0;
    __syncthreads();
    int mine = -1;
    for (int c0 = 0; c0 < a.pairs; c0 += 8 * 1024) {
        int64_t id[8];                             // in flight at once
#pragma unroll
        for (int i = 0; i < 8; ++i) id[i] = a.idx[min(c0 + i * 1024 + tid, a.pairs - 1)];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 / 1024 + i, e = c * 1024 + tid < a.pairs ? local_id(a, id[i]) : -1;
            if (c == own) mine = e;
            if (e >= 0) atomicAdd(&(c < own ? before : c > own ? behind : lds + wave * a.experts)[e], 1);
        }
    }
    __syncthreads();
    // thread e: the expert's total (experts <= 512), then an exclusive prefix over the experts
    int count = 0, earlier = 0;
    if (tid < a.experts) {
        earlier = before[tid];
        count = earlier + behind[tid];
#pragma unroll
        for (int w = 0; w < 16; ++w) count += lds[w * a.experts + tid];
    }
    const int incl = wave_prefix(count, lane);
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    int first = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        const int v = sums[w];
        first += w < wave ? v : 0;
        all += v;
    }
    if (tid < a.experts) {
        const int start = first + incl - count;
        if (own == 0) a.offsets[tid] = start;
        int at = start + earlier;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const int c = lds[w * a.experts + tid];
            lds[w * a.experts + tid] = at;
            at += c;
        }
    }
    if (own == 0 && tid == 0) a.offsets[a.experts] = all;
    __syncthreads();
    place_pairs(a, mine, p, a.pairs, lds + wave * a.experts, bits_of(a.experts));
    if (p >= all && p < a.pairs) a.order[p] = -1;
}

// Many pairs, three launches.  1: every chunk's counts, hist[expert][chunk].  Dynamic LDS: int [experts].
__global__ __launch_bounds__(256) void order_count_kernel(OrderArgs a) {
    extern __shared__ int lds[];
    for (int i = threadIdx.x; i < a.experts; i += 256) lds[i] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.per_chunk, hi = min(lo + a.per_chunk, (int64_t)a.pairs);
#pragma unroll 4
    for (int64_t p = lo + threadIdx.x; p < hi; p += 256) {
        const int e = local_of(a, (int)p);
        if (e >= 0) atomicAdd(&lds[e], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.experts; i += 256) a.hist[(size_t)i * a.chunks + blockIdx.x] = lds[i];
}

// 2: one wave per expert: its chunks' counts become their first places within the expert, and its total.
__global__ __launch_bounds__(256) void order_scan_kernel(OrderArgs a) {
    const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (e >= a.experts) return;
    int32_t* h = a.hist + (size_t)e * a.chunks;
    int run = 0;
    for (int c = lane; c - lane < a.chunks; c += 64) {
        const int v = c < a.chunks ? h[c] : 0;
        const int incl = wave_prefix(v, lane);
        if (c < a.chunks) h[c] = run + incl - v;
        run += __shfl(incl, 63);
    }
    if (lane == 0) a.hist[(size_t)a.experts * a.chunks + e] = run;
}

// 3: places.  Every work-group adds up the experts' totals for their first places.  Dynamic LDS: int [4][experts],
// then int [4].
// kShort: a wave has at most kPairsPerWave pairs, whose ids stay in registers (262144 pairs: 7.4 us against 8.0).
template <bool kShort>
__global__ __launch_bounds__(256) void order_place_kernel(OrderArgs a) {
    extern __shared__ int lds[];
    int* sums = lds + 4 * a.experts;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t first = (int64_t)blockIdx.x * a.per_chunk;
    const int per = a.per_chunk / 4;
    const int64_t end = min(first + a.per_chunk, (int64_t)a.pairs);
    const int lo = (int)min(first + (int64_t)wave * per, end), hi = (int)min((int64_t)lo + per, end);
    constexpr int kMine = kShort ? kPairsPerWave / 64 : 1;
    int mine[kMine];
    if constexpr (kShort)
#pragma unroll
        for (int i = 0; i < kMine; ++i) mine[i] = lo + i * 64 + lane < hi ? local_of(a, lo + i * 64 + lane) : -1;
    // the first batch of experts' places, on their way while the pairs are counted
    const int* totals = a.hist + (size_t)a.experts * a.chunks;
    int before = tid < a.experts ? a.hist[(size_t)tid * a.chunks + blockIdx.x] : 0, count = tid < a.experts ? totals[tid] : 0;
    for (int i = tid; i < 4 * a.experts; i += 256) lds[i] = 0;
    __syncthreads();
    if constexpr (kShort) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (mine[i] >= 0) atomicAdd(&lds[wave * a.experts + mine[i]], 1);
    } else {
#pragma unroll 4
        for (int p = lo + lane; p < hi; p += 64) {
            const int e = local_of(a, p);
            if (e >= 0) atomicAdd(&lds[wave * a.experts + e], 1);
        }
    }
    int base = 0;                                  // pairs of the experts before this batch of 256
    for (int e0 = 0; e0 < a.experts; e0 += 256) {
        const int e = e0 + tid;
        if (e0) {
            before = e < a.experts ? a.hist[(size_t)e * a.chunks + blockIdx.x] : 0;
            count = e < a.experts ? totals[e] : 0;
        }
        const int incl = wave_prefix(count, lane);
        if (lane == 63) sums[wave] = incl;
        __syncthreads();
        int start = base + incl - count, all = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int v = sums[w];
            start += w < wave ? v : 0;
            all += v;
        }
        if (e < a.experts) {
            if (blockIdx.x == 0) a.offsets[e] = start;
            int at = start + before;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int c = lds[w * a.experts + e];
                lds[w * a.experts + e] = at;
                at += c;
            }
        }
        base += all;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = base;
    const int bits = bits_of(a.experts);
    if constexpr (kShort) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (lo + i * 64 < hi) place_pairs(a, mine[i], lo + i * 64 + lane, hi, lds + wave * a.experts, bits);
    } else {
        for (int p0 = lo; p0 < hi; p0 += 64)
            place_pairs(a, p0 + lane < hi ? local_of(a, p0 + lane) : -1, p0 + lane, hi, lds + wave * a.experts, bits);
    }
    for (int64_t i = max(first, (int64_t)base) + tid; i < end; i += 256) a.order[i] = -1;
}

// The three-launch form: pairs per work-group, a multiple of 4 waves x 64, and at most 1024 chunks of that many.  No
// pairs are one empty chunk, whose launches write the offsets; the workspace is sized for the same count.
struct Chunks {
    int per, count;
    uint64_t bytes(int experts) const { return (uint64_t)(count + 1) * experts * 4; }     // and the experts' totals
};
Chunks chunks_of(int64_t pairs) {
    const int64_t least = 4 * kPairsPerWave, by_chunks = (pairs + 1023) / 1024;
    const int64_t per = ((by_chunks < least ? least : by_chunks) + 255) / 256 * 256, count = (pairs + per - 1) / per;
    return Chunks{(int)per, (int)(count > 0 ? count : 1)};
}
bool few_pairs(int64_t pairs, int experts) { return pairs <= kFewPairs && experts <= kFewExperts; }

int32_t check_router(const mega_moe_router_config* c) {
    if (!c || c->tokens < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (c->num_experts < 1 || c->num_experts > MEGA_MOE_MAX_EXPERTS || c->topk < 1 || c->topk > MEGA_MOE_MAX_TOPK ||
        c->topk > c->num_experts || c->tokens > MEGA_MOE_MAX_PAIRS || c->tokens * c->topk > MEGA_MOE_MAX_PAIRS ||
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

uint32_t router_grid(int64_t tokens, int per) {
    const int64_t g = (tokens + per - 1) / per;
    return (uint32_t)(g < (1 << 20) ? g : 1 << 20);
}

template <int EPL, int LANES, bool kSigmoid, class Key, bool kGroups>
hipError_t launch_router(const RouterArgs& a, hipStream_t st) {
    // the groups' values take EPL * 512 bytes of LDS per wave
    constexpr int WAVES = kGroups && EPL > 16 ? 1 : 4;
    hipLaunchKernelGGL((router_kernel<EPL, LANES, kSigmoid, Key, kGroups, WAVES>),
                       dim3(router_grid(a.tokens, WAVES * 64 / LANES)), dim3(WAVES * 64), 0, st, a);
    return hipGetLastError();
}
template <int EPL, int LANES, class Key>
hipError_t pick_form(const RouterArgs& a, bool sigmoid, hipStream_t st) {
    switch ((sigmoid ? 2 : 0) | (a.G > 1 ? 1 : 0)) {
        case 0: return launch_router<EPL, LANES, false, Key, false>(a, st);
        case 1: return launch_router<EPL, LANES, false, Key, true>(a, st);
        case 2: return launch_router<EPL, LANES, true, Key, false>(a, st);
        default: return launch_router<EPL, LANES, true, Key, true>(a, st);
    }
}
template <int EPL, int LANES>
hipError_t pick_router(const RouterArgs& a, bool sigmoid, hipStream_t st) {
    if constexpr (EPL <= 16) {
        if (!a.bias && a.type == MEGA_MOE_FP32) return pick_form<EPL, LANES, double>(a, sigmoid, st);
        if (!a.bias) return pick_form<EPL, LANES, uint32_t>(a, sigmoid, st);
    }
    return pick_form<EPL, LANES, uint64_t>(a, sigmoid, st);
}
template <int EPL, int LANES>
hipError_t pick_backward(const RouterArgs& a, bool sigmoid, hipStream_t st) {
    constexpr int WAVES = EPL > 16 ? 1 : 4;
    const dim3 grid(router_grid(a.tokens, WAVES * 64 / LANES)), block(WAVES * 64);
    if (sigmoid) hipLaunchKernelGGL((router_backward_kernel<EPL, LANES, true, false, WAVES>), grid, block, 0, st, a);
    else if (a.renorm) hipLaunchKernelGGL((router_backward_kernel<EPL, LANES, false, false, WAVES>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((router_backward_kernel<EPL, LANES, false, true, WAVES>), grid, block, 0, st, a);
    return hipGetLastError();
}
// A quarter wave per token: enough tokens to fill the CUs with them (4 waves to a SIMD), and room in 16 lanes.
bool by_quarters(const RouterArgs& a) { return a.tokens >= 4096 && a.E <= 256 && a.K <= 16 && a.G <= 16; }

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
    const hipError_t e = by_quarters(a) ? (a.E <= 64    ? pick_router<4, 16>(a, sigmoid, st)
                                           : a.E <= 128 ? pick_router<8, 16>(a, sigmoid, st)
                                                        : pick_router<16, 16>(a, sigmoid, st))
                         : a.E <= 64   ? pick_router<1, 64>(a, sigmoid, st)
                         : a.E <= 128  ? pick_router<2, 64>(a, sigmoid, st)
                         : a.E <= 256  ? pick_router<4, 64>(a, sigmoid, st)
                         : a.E <= 512  ? pick_router<8, 64>(a, sigmoid, st)
                         : a.E <= 1024 ? pick_router<16, 64>(a, sigmoid, st)
                                       : pick_router<64, 64>(a, sigmoid, st);
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
    const hipError_t e = by_quarters(a) ? (a.E <= 64    ? pick_backward<4, 16>(a, sigmoid, st)
                                           : a.E <= 128 ? pick_backward<8, 16>(a, sigmoid, st)
                                                        : pick_backward<16, 16>(a, sigmoid, st))
                         : a.E <= 64   ? pick_backward<1, 64>(a, sigmoid, st)
                         : a.E <= 128  ? pick_backward<2, 64>(a, sigmoid, st)
                         : a.E <= 256  ? pick_backward<4, 64>(a, sigmoid, st)
                         : a.E <= 512  ? pick_backward<8, 64>(a, sigmoid, st)
                         : a.E <= 1024 ? pick_backward<16, 64>(a, sigmoid, st)
                                       : pick_backward<64, 64>(a, sigmoid, st);
    return e == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

int32_t mega_moe_group_workspace_bytes(int64_t pairs, int32_t num_local_experts, uint64_t* bytes_out) {
    if (!bytes_out || pairs < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (pairs > MEGA_MOE_MAX_PAIRS || num_local_experts < 1 || num_local_experts > MEGA_MOE_MAX_EXPERTS)
        return MEGA_MOE_ERR_UNSUPPORTED;
    *bytes_out = few_pairs(pairs, num_local_experts) ? 0 : chunks_of(pairs).bytes(num_local_experts);
    return MEGA_MOE_OK;
}

int32_t mega_moe_group_by_expert(const int64_t* topk_idx, int64_t pairs, int32_t first_expert,
                                 int32_t num_local_experts, int32_t* offsets, int32_t* order, int32_t* slot,
                                 void* workspace, uint64_t workspace_bytes, void* stream) {
    uint64_t need = 0;
    const int32_t rc = mega_moe_group_workspace_bytes(pairs, num_local_experts, &need);
    if (rc) return rc;
    if (first_expert < 0) return MEGA_MOE_ERR_INVALID_ARG;
    if (!aligned16(offsets) || (need && !aligned16(workspace)) ||
        (pairs > 0 && (!aligned16(topk_idx) || !aligned16(order) || !aligned16(slot))))
        return MEGA_MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MEGA_MOE_ERR_WORKSPACE_TOO_SMALL;
    hipStream_t st = static_cast<hipStream_t>(stream);
    OrderArgs a{topk_idx, offsets, order, slot, static_cast<int32_t*>(workspace), (int)pairs, first_expert,
                num_local_experts, 0, 0};
    if (few_pairs(pairs, num_local_experts)) {
        hipLaunchKernelGGL(order_few_kernel, dim3((uint32_t)(pairs > 1024 ? (pairs + 1023) / 1024 : 1)), dim3(1024),
                           (18 * num_local_experts + 32) * sizeof(int), st, a);
        return hipGetLastError() == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
    }
    const Chunks c = chunks_of(pairs);
    a.per_chunk = c.per;
    a.chunks = c.count;
    const dim3 chunks(a.chunks), block(256);
    hipLaunchKernelGGL(order_count_kernel, chunks, block, num_local_experts * sizeof(int), st, a);
    hipLaunchKernelGGL(order_scan_kernel, dim3((num_local_experts + 3) / 4), block, 0, st, a);
    const size_t lds = (4 * num_local_experts + 4) * sizeof(int);
    if (a.per_chunk <= 4 * kPairsPerWave) hipLaunchKernelGGL(order_place_kernel<true>, chunks, block, lds, st, a);
    else hipLaunchKernelGGL(order_place_kernel<false>, chunks, block, lds, st, a);
    return hipGetLastError() == hipSuccess ? MEGA_MOE_OK : MEGA_MOE_ERR_HIP;
}

}  // extern "C"
