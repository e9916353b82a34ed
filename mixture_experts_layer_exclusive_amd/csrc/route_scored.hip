// Routing by scores, with a balance bias and groups of experts, and its gradient.
//
//   s[t, e]  = sigmoid(l[t, e]), or softmax over the experts
//   c[t, e]  = s[t, e] + bias[e]             (the order of choice, not the gates)
//   group    value: the sum of its group_top largest c; the groups_kept best stay
//   ids      the k largest c of the groups that stay, ties to the lower expert
//   gates    scale * s of the chosen, over the sum of the chosen s if renormalised
//
// c decides between experts, so it is defined in 64 bits: two scores that differ in
// the 30th bit are in the right order.  Without a bias c has the order of the
// logits, which then stand for it (unless groups are valued by sums).
//
// For k <= 16 the choice is made in 32 bits by G lanes per token, and where it hangs
// on a difference that 32 bits may have got wrong, the whole wave makes that token's choice
// again in 64 bits.  How often depends on the logits: with a bias about one token in 1000;
// by groups valued by sums without one, where scores near their end (1, or 0) are alike,
// most tokens of wide logits.  32768 x 256 in 8 groups of which 4 stay, k = 8, normal logits
// of standard deviation 2, 4, 6, 8: sigmoid 0.3, 11, 95 and 100 % of the tokens, 27, 48, 100
// and 98 us; softmax 0.2, 1.3, 10 and 28 %, 26, 32, 49 and 70 us; with a bias 24 to 26 us all.
// Equal scores that compete always go there.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "device_util.h"
#include "moe_internal.h"
#include "scored_plan.h"

namespace moe {

namespace {

constexpr int kEpl = MOE_MAX_EXPERTS / 64;  // experts per lane of a whole wave: lane, lane + 64, ..

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Whether (v, e) is chosen before (w, f).
__device__ __forceinline__ bool before(double v, int e, double w, int f) { return v > w || (v == w && e < f); }

// LDS that a wave writes and reads by itself, in the order of the source (also where
// the types differ).
__device__ __forceinline__ void wave_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// ---- values that carry their index ------------------------------------------------
//
// A key is a 64-bit float: a 32-bit c, with the index in the low bits such that of equal
// c the lower index is the larger key (below zero a larger fraction is a smaller
// number).  Then the larger of two keys is one instruction, index and all.

__device__ __forceinline__ double key_max(double a, double b) {
    double d;  // (fmax would quiet signalling NaNs first: there are none)
    asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double key_min(double a, double b) {
    double d;
    asm("v_min_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double key_of(uint32_t hi, int e) {
    const uint32_t sign = static_cast<uint32_t>(static_cast<int32_t>(hi) >> 31);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | (sign ^ static_cast<uint32_t>(255 - e)));
}
__device__ __forceinline__ int key_index(double key) {
    const uint64_t b = __builtin_bit_cast(uint64_t, key);
    return 255 - static_cast<int>(static_cast<uint32_t>(b) ^ static_cast<uint32_t>(static_cast<int64_t>(b) >> 63));
}
__device__ __forceinline__ float key_value(double key) {
    return __uint_as_float(static_cast<uint32_t>(__builtin_bit_cast(uint64_t, key) >> 32));
}
// Upper halves: of c (any float's bits are those of a finite 64-bit one; a NaN comes
// last, -0 is 0), and of what is out, below minus infinity.
__device__ __forceinline__ uint32_t key_high(float c) { return __float_as_uint(fmaxf(c + 0.f, -INFINITY)); }
constexpr uint32_t kOut = 0xffefffffu;

// ---- within the G lanes of a token ---------------------------------------------------
//
// Each step pairs a lane with one of the other half of the lanes that hold the same by
// then: neighbours, pairs, and the mirror images within 8 and 16 lanes.
constexpr int kStep[4] = {0xB1, 0x4E, 0x141, 0x140};
template <int G>
constexpr int kSteps = G == 4 ? 2 : (G == 8 ? 3 : 4);

template <int STEP>
__device__ __forceinline__ int partner(int v) {
    return __builtin_amdgcn_update_dpp(0, v, kStep[STEP], 0xf, 0xf, true);
}
template <int STEP>
__device__ __forceinline__ float partner(float v) {
    return __builtin_bit_cast(float, partner<STEP>(__builtin_bit_cast(int, v)));
}
template <int STEP>
__device__ __forceinline__ double partner(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = partner<STEP>(static_cast<int>(b)), hi = partner<STEP>(static_cast<int>(b >> 32));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// The token's lanes turned by I (which way does not matter to who takes all turns).
template <int G, int I>
__device__ __forceinline__ int turned(int v) {
    if constexpr (G == 16) return __builtin_amdgcn_update_dpp(0, v, 0x120 + I, 0xf, 0xf, true);
    else if constexpr (G == 4)
        return __builtin_amdgcn_update_dpp(0, v, I | ((1 + I) & 3) << 2 | ((2 + I) & 3) << 4 | ((3 + I) & 3) << 6, 0xf, 0xf, true);
    else return __shfl(v, (lane_id() & ~(G - 1)) | ((lane_id() + I) & (G - 1)), 64);
}
// How many of the token's other lanes (every STEP-th) have a larger key.
template <int G, int STEP, int I = STEP>
__device__ __forceinline__ int larger_keys(double key) {
    if constexpr (I >= G) return 0;
    else {
        const uint64_t b = __builtin_bit_cast(uint64_t, key);
        const uint32_t lo = turned<G, I>(static_cast<int>(b)), hi = turned<G, I>(static_cast<int>(b >> 32));
        return (__builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo) > key ? 1 : 0) +
               larger_keys<G, STEP, I + STEP>(key);
    }
}
template <int G, typename T, typename F>
__device__ __forceinline__ T reduce(T v, F op) {
    v = op(v, partner<0>(v));
    v = op(v, partner<1>(v));
    if constexpr (G >= 8) v = op(v, partner<2>(v));
    if constexpr (G >= 16) v = op(v, partner<3>(v));
    return v;
}
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Min {
    __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct Add {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// ---- sorted lists of KM keys, the largest first ---------------------------------------

__device__ __forceinline__ void order(double& a, double& b) {
    const double x = key_max(a, b);
    b = key_min(a, b);
    a = x;
}
__device__ __forceinline__ void sort4(double* v) {
    order(v[0], v[1]); order(v[2], v[3]);
    order(v[0], v[2]); order(v[1], v[3]);
    order(v[1], v[2]);
}
// (19 comparisons: Batcher's odd-even merge sort)
__device__ __forceinline__ void sort8(double* v) {
    sort4(v);
    sort4(v + 4);
    order(v[0], v[4]); order(v[1], v[5]); order(v[2], v[6]); order(v[3], v[7]);
    order(v[2], v[4]); order(v[3], v[5]);
    order(v[1], v[2]); order(v[3], v[4]); order(v[5], v[6]);
}
// Sorts keys that first rise and then fall, or the other way.
template <int KM>
__device__ __forceinline__ void straighten(double* a) {
#pragma unroll
    for (int d = KM / 2; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < KM; ++i)
            if ((i & d) == 0) order(a[i], a[i + d]);
}
// The KM largest of a and b, sorted: with b the other way round the larger of each pair
// are they.
template <int KM>
__device__ __forceinline__ void merge(double* a, const double* b) {
#pragma unroll
    for (int i = 0; i < KM; ++i) a[i] = key_max(a[i], b[KM - 1 - i]);
    straighten<KM>(a);
}
template <int STEP, int KM>
__device__ __forceinline__ void merge_partner(double* a) {
    double b[KM];
#pragma unroll
    for (int i = 0; i < KM; ++i) b[i] = partner<STEP>(a[i]);
    merge<KM>(a, b);
}
// A lane's EPL keys: the KM largest of them, sorted (fewer: the list has room after them).
template <int KM, int EPL>
__device__ __forceinline__ void sort_lane(double* v) {
    static_assert(EPL == 8 || EPL == 16, "experts per lane");
    if constexpr (KM == 4) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) sort4(v + i);
#pragma unroll
        for (int i = 4; i < EPL; i += 4) merge<4>(v, v + i);
    } else {
        sort8(v);
        if constexpr (EPL == 16) {
            sort8(v + 8);
            if constexpr (KM == 8) {
                merge<8>(v, v + 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const double x = v[8 + i];
                    v[8 + i] = v[15 - i];
                    v[15 - i] = x;
                }
                straighten<16>(v);
            }
        }
    }
}

// ---- a token's choice in 64 bits, by a whole wave ---------------------------------------

// buf: 2 * MOE_MAX_EXPERTS doubles of LDS.  `l`, `s`: of the lane's experts.
__device__ __forceinline__ void choose64(const moe_gating_t& g, const float* __restrict__ logits,
                                         const float* __restrict__ bias, int64_t t, double* buf,
                                         int32_t* __restrict__ ids, float* __restrict__ gates, double (&s)[kEpl]) {
    const int lane = lane_id();
    const int E = g.E, k = g.k;
    const int size = E / g.groups;
    const bool limited = g.groups_kept < g.groups;
    const bool by_logit = bias == nullptr && (!limited || g.group_top == 1);
    double l[kEpl], c[kEpl];
    double top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
        const int e = lane + 64 * j;
        l[j] = e < E ? logits[t * E + e] : -INFINITY;
        top = fmax(top, l[j]);
    }
    if (g.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = fmax(top, __shfl_xor(top, off, 64));
        double z = 0;
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            // (a row of minus infinities: all scores zero)
            s[j] = top == -INFINITY || lane + 64 * j >= E ? 0 : exp(l[j] - top);
            z += s[j];
        }
        z = wave_sum(z);
#pragma unroll
        for (int j = 0; j < kEpl; ++j) s[j] = z == 0 ? 0 : s[j] / z;
    } else {
#pragma unroll
        for (int j = 0; j < kEpl; ++j) s[j] = lane + 64 * j < E ? 1.0 / (1.0 + exp(-l[j])) : 0;
    }
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
        const int e = lane + 64 * j;
        c[j] = by_logit ? l[j] : s[j] + (bias != nullptr && e < E ? bias[e] : 0.f);
        // (a NaN comes last; an expert that is out has -DBL_MAX, below any that is not)
        c[j] = c[j] == c[j] ? fmin(fmax(c[j], -1e308), 1e308) : -1e308;
        if (e >= E) c[j] = -DBL_MAX;
    }
    if (limited) {
        double* const c_of = buf;
        double* const v_of = buf + MOE_MAX_EXPERTS;
#pragma unroll
        for (int j = 0; j < kEpl; ++j)
            if (lane + 64 * j < E) c_of[lane + 64 * j] = c[j];
        wave_lds();
        for (int q = lane; q < g.groups; q += 64) {
            double a = -DBL_MAX, b = -DBL_MAX;
#pragma unroll 8
            for (int e = q * size; e < (q + 1) * size; ++e) {
                const double v = c_of[e];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
            // (a sum with an infinity is that, a sum of both is a NaN and comes last)
            const double sum = a >= 1e308 && b <= -1e308 ? -1e308 : fmin(fmax(a + b, -1e308), 1e308);
            v_of[q] = g.group_top == 2 && size > 1 ? sum : a;
        }
        wave_lds();
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            const int e = lane + 64 * j;
            if (e >= E) continue;
            const int mine = e / size;
            int rank = 0;
#pragma unroll 8
            for (int q = 0; q < g.groups; ++q) rank += before(v_of[q], q, v_of[mine], mine) ? 1 : 0;
            if (rank >= g.groups_kept) c[j] = -DBL_MAX;
        }
        wave_lds();
    }
    double my_s = 0;
    int my_e = 0;
    for (int r = 0; r < k; ++r) {
        double m = c[0];
#pragma unroll
        for (int j = 1; j < kEpl; ++j) m = key_max(m, c[j]);
        m = reduce<16>(m, [](double a, double b) { return key_max(a, b); });
        const uint64_t bits = __builtin_bit_cast(uint64_t, m);
        double row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(bits), 16 * i);
            const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(bits >> 32), 16 * i);
            row[i] = __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
        }
        m = key_max(key_max(row[0], row[1]), key_max(row[2], row[3]));
        // the lowest expert that has it
        int e = 0;
#pragma unroll
        for (int j = kEpl - 1; j >= 0; --j) {
            const uint64_t has = __ballot(c[j] == m);
            if (has != 0) e = 64 * j + __builtin_ctzll(has);
        }
        double ws = s[0];
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            if (e >> 6 == j) {
                ws = s[j];
                if (lane == (e & 63)) c[j] = -DBL_MAX;
            }
        }
        ws = __shfl(ws, e & 63, 64);
        if (lane == r) {
            my_s = ws;
            my_e = e;
        }
    }
    double total = wave_sum(my_s);
    // Scores that vanish even here have the shares of exp(l - most), as 1 - s is 1; but
    // sigmoid scores that are 0 in 64 bits (logits masked by the type's lowest value) stay 0.
    if (g.renormalise && total < 0x1p-800 && (total > 0 || g.score == MOE_SCORE_SOFTMAX)) {
        const double mine = lane < k ? logits[t * E + my_e] : -INFINITY;
        double most = mine;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) most = fmax(most, __shfl_xor(most, off, 64));
        my_s = most == -INFINITY ? 0 : exp(mine - most);
        total = wave_sum(my_s);
    }
    if (lane < k) {
        ids[t * k + lane] = my_e;
        const double v = g.renormalise ? (total == 0 ? 0 : my_s / total) : my_s;
        gates[t * k + lane] = static_cast<float>(g.scale * v);
    }
}

// Any k: a wave per token, its share of the tokens one after the other.
__global__ __launch_bounds__(256) void route_scored_wave_kernel(moe_gating_t g, const float* __restrict__ logits,
                                                               const float* __restrict__ bias,
                                                               int32_t* __restrict__ ids, float* __restrict__ gates,
                                                               float* __restrict__ partial) {
    __shared__ double s_buf[4][2 * MOE_MAX_EXPERTS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double sum[kEpl] = {};
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < g.T; t += static_cast<int64_t>(gridDim.x) * 4) {
        double s[kEpl];
        choose64(g, logits, bias, t, s_buf[wave], ids, gates, s);
#pragma unroll
        for (int j = 0; j < kEpl; ++j) sum[j] += s[j];
    }
    if (partial == nullptr) return;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEpl; ++j) s_buf[wave][lane + 64 * j] = sum[j];
    __syncthreads();
    const int e = threadIdx.x;
    if (e < g.E)
        partial[static_cast<int64_t>(blockIdx.x) * g.E + e] =
            static_cast<float>((s_buf[0][e] + s_buf[1][e]) + (s_buf[2][e] + s_buf[3][e]));
}

// ---- a token's choice in 32 bits, by G lanes ------------------------------------------------
//
// Lane s of a token has the EPL experts from EPL * s on.  Each lane sorts its KM >= k
// largest keys, and the lists are merged over the lanes.  Groups that are whole lanes (a
// power of two of them) are valued by the heads of the lists, and the lists of groups that
// go are dropped; other groups are valued from LDS before the lists are made.
//
// Errors, u = 2^-24.  Sigmoid: exp2 of the rounded product l log2(e) is off by (|l| + 2) u
// of itself, which counts s (1 - s) times in s, and |l| s (1 - s) < 1 / 4; the sum and the
// reciprocal add 3 u s: together below 4 u, 8 u for a difference of two.  Softmax: (2 |l - max|
// + 2) u of s, where |l - max| s < max s, and the quotient 1 u; its sum's error, 20 roundings
// and its terms' own (2 |l - max| + 2, below 9 in the mean over the scores of 256 experts),
// 30 u, is the same share of all of a token's s, so it counts once in a difference: 30 u + 2 *
// 5 u of max s, below 2^-18.6.  The sum with the bias adds 2 u |c| to a difference.  A choice
// is taken for certain if all that it compared differs by more than 2^-20 (softmax: 2^-18 max
// s) + 2^-22 max |c|, twice that for groups (sums of two), else it is made again in 64 bits.
//
// Bound by instructions (about 1000 for the 4 tokens of a wave, a third of them the lists'),
// not by the logits' bytes: 32768 tokens, 256 experts, k = 8: 15 us by logits or scores (6 us
// for the bytes at a copy's rate), 20 with a bias, 26 in 8 groups, of which 4 the certainty's
// checks and a few tokens' second choice, and 27 with partial score sums, whose adding takes
// 4; one token 5.3 us.  A whole wave per token in 64 bits took 161 us.  Of 16 experts per lane
// 2 to 5 values are spilled, and where E is no multiple of 4 the row lies in scratch memory
// (load_experts).
constexpr int kMaxRounds = 32;  // of tokens that a workgroup takes one after the other
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLeastLogit = -709.78f;  // sigmoid scores of lower ones are 0 in 64 bits: exp(-l) overflows

typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));

// Values e0 .. e0 + EPL - 1 of a row of E >= 4, in 16-byte loads whatever the row's
// alignment (4-byte loads: 250 experts 48 us for 36).  The last load of a row ends with it;
// unless E is a multiple of 4 (VEC), what it holds is moved down, which the compiler makes
// an indexed read of the array: it lies in scratch memory (48 to 96 bytes per lane), and 250
// experts take 39 us where 256 take 23 (39008 tokens, a bias, k = 8).  Values past the row are
// any.
template <int EPL, bool VEC>
__device__ __forceinline__ void load_experts(const float* __restrict__ row, int e0, int E, float (&v)[EPL]) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const f32x4_any_t w = *reinterpret_cast<const f32x4_any_t*>(row + min(e0 + i, E - 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = w[j];
    }
    if (!VEC && e0 + EPL > E) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            const int by = e0 + i - (E - 4);  // 1, 2, 3: the row ends in this load
            if (by > 0 && by < 4) {
                v[i] = by == 1 ? v[i + 1] : (by == 2 ? v[i + 2] : v[i + 3]);
                v[i + 1] = by == 1 ? v[i + 2] : v[i + 3];
                v[i + 2] = v[i + 3];
            }
        }
    }
}

template <int G, int EPL, bool VEC, int KM>
__global__ __launch_bounds__(256, KM == 16 || (EPL == 16 && !VEC) ? 3 : 4) void route_scored_kernel(moe_gating_t g, const float* __restrict__ logits,
                                                          const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                          float* __restrict__ gates, float* __restrict__ partial) {
    constexpr int TPW = 64 / G;              // tokens per wave
    constexpr int EMAX = G * EPL;
    // a wave's LDS: c and the groups' values of its tokens, or choose64's, or (of all
    // waves together) the score sums
    constexpr int BUF = TPW * EMAX > 2 * MOE_MAX_EXPERTS ? TPW * EMAX : 2 * MOE_MAX_EXPERTS;
    __shared__ double s_buf[4][BUF];
    __shared__ uint64_t s_again[4][kMaxRounds];
    // the bias, where its loads would have to be moved as the logits' are (39008 tokens, 250
    // experts: 50 us for 40)
    __shared__ alignas(16) float s_bias[VEC ? 4 : EMAX];
    if (!VEC && bias != nullptr) {
        for (int e = threadIdx.x; e < EMAX; e += 256) s_bias[e] = e < g.E ? bias[e] : 0.f;
        __syncthreads();
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane / G, s_lane = lane % G;
    const int E = g.E, k = g.k;
    const int size = E / g.groups;
    const bool limited = g.groups_kept < g.groups;
    const bool by_logit = bias == nullptr && (!limited || g.group_top == 1);
    const int per_group = size / EPL;        // lanes of a group
    const bool whole_lanes = limited && size % EPL == 0 && (per_group & (per_group - 1)) == 0;
    const int e0 = s_lane * EPL;
    float sum[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum[i] = 0.f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 4 * TPW;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * TPW;
    int round = 0;                           // (at most kMaxRounds)
    for (int64_t t0 = first; t0 < g.T; t0 += step, ++round) {
        const bool has = t0 + row < g.T;
        // (lanes past the last token work on it once more and store nothing)
        const int64_t t = has ? t0 + row : g.T - 1;
        const float* const from = logits + t * E;
        float c[EPL], s[EPL];
        uint32_t gone = ~0u << min(max(E - e0, 0), EPL);  // bit i: expert e0 + i is out
        asm volatile("" : "+v"(gone));       // (keeps masks made of it out of scalar registers)
        load_experts<EPL, VEC>(from, e0, E, c);
        // (experts past the last: minus infinity)
        if (e0 + EPL > E) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = gone >> i & 1 ? -INFINITY : c[i];
        }
        // scores (experts past the last: zero)
        float top = -INFINITY, inv = 1.f, s_error = 0x1p-20f;
        if (g.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) top = fmaxf(top, c[i]);
            top = reduce<G>(top, Max());
            const float shift = top == -INFINITY ? 0.f : top;
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                s[i] = __builtin_amdgcn_exp2f((c[i] - shift) * kLog2e);
                z += s[i];
            }
            z = reduce<G>(z, Add());
            inv = z == 0.f ? 0.f : 1.f / z;
            s_error = 0x1p-18f * inv;  // (the largest s is 1 / z)
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] *= inv;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-c[i] * kLog2e));
        }
        if (partial != nullptr && has) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) sum[i] += s[i];
        }
        if (!by_logit) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = s[i];
            if (bias != nullptr) {
                float b[EPL];
                if constexpr (VEC) {
                    load_experts<EPL, VEC>(bias, e0, E, b);
                } else {
#pragma unroll
                    for (int i = 0; i < EPL; ++i) b[i] = s_bias[e0 + i];
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i) c[i] += b[i];
            }
            // (again: neither a score of zero nor what was loaded past the bias is near a choice)
            if (e0 + EPL > E) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) c[i] = gone >> i & 1 ? -INFINITY : c[i];
            }
        }
        bool sure = true;
        bool dropped = false;                // the lane's experts are out
        float* const c_of = reinterpret_cast<float*>(s_buf[wave]) + row * EMAX;
        float* const v_of = reinterpret_cast<float*>(s_buf[wave]) + TPW * EMAX + row * EMAX;
        // the groups that stay differ from those that go by more than the error
        auto apart = [&](float low, float high, float most) {
            low = reduce<G>(low, Min());
            high = reduce<G>(high, Max());
            most = reduce<G>(most, Max());
            return low - high > 2.f * (s_error + 0x1p-22f * most);
        };
        if (limited && !whole_lanes) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e0 + i < E) c_of[e0 + i] = c[i] == c[i] ? c[i] : -INFINITY;
            wave_lds();
            float most = 0.f;
            for (int q = s_lane; q < g.groups; q += G) {
                float a = -INFINITY, a2 = -INFINITY;
#pragma unroll 8
                for (int i = 0; i < size; ++i) {
                    const float v = c_of[q * size + i];
                    a2 = fmaxf(a2, fminf(a, v));
                    a = fmaxf(a, v);
                }
                const float v = g.group_top == 2 && size > 1 ? a + a2 : a;
                v_of[q] = v == v ? v : -INFINITY;
                most = fmaxf(most, fmaxf(fabsf(a), size > 1 ? fabsf(a2) : 0.f));
            }
            wave_lds();
            float low = INFINITY, high = -INFINITY;
            uint32_t stay[(EMAX + 32 * G - 1) / (32 * G)] = {};   // bit i: group s_lane + G * i
            int n = 0;
            for (int q = s_lane; q < g.groups; q += G, ++n) {
                const float v = v_of[q];
                int rank = 0;
#pragma unroll 8
                for (int o = 0; o < g.groups; ++o) rank += v_of[o] > v || (v_of[o] == v && o < q) ? 1 : 0;
                if (rank < g.groups_kept) {
                    stay[n / 32] |= 1u << (n & 31);
                    low = fminf(low, v);
                } else {
                    high = fmaxf(high, v);
                }
            }
            wave_lds();
            n = 0;
            for (int q = s_lane; q < g.groups; q += G, ++n) v_of[q] = stay[n / 32] >> (n & 31) & 1 ? 1.f : 0.f;
            wave_lds();
            int q = e0 / size, r = e0 - q * size;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if (v_of[min(q, g.groups - 1)] == 0.f) {
                    gone |= 1u << i;
                    c[i] = -INFINITY;
                }
                if (++r == size) {
                    r = 0;
                    ++q;
                }
            }
            wave_lds();
            if (!by_logit) sure = apart(low, high, most);
        }
        double list[EPL > KM ? EPL : KM];
#pragma unroll
        for (int i = 0; i < EPL; ++i) list[i] = key_of(gone >> i & 1 ? kOut : key_high(c[i]), e0 + i);
        sort_lane<KM, EPL>(list);
#pragma unroll
        for (int i = EPL; i < KM; ++i) list[i] = key_of(kOut, 255);
        if (whole_lanes) {
            // the group's two largest, from the lists' heads
            const bool live = e0 < E;
            float a = live ? key_value(list[0]) : -INFINITY, a2 = live ? key_value(list[1]) : -INFINITY;
            auto join = [&](float p, float p2) {
                a2 = fmaxf(fminf(a, p), fmaxf(a2, p2));
                a = fmaxf(a, p);
            };
            if (per_group >= 2) join(partner<0>(a), partner<0>(a2));
            if (per_group >= 4) join(partner<1>(a), partner<1>(a2));
            if constexpr (G >= 8) {
                if (per_group >= 8) join(partner<2>(a), partner<2>(a2));
            }
            float v = g.group_top == 2 ? a + a2 : a;
            // (the group's number, counted from the token's first lane)
            const int q = s_lane / per_group;
            v = __uint_as_float(key_high(v));
            const double mine = key_of(live ? __float_as_uint(v) : kOut, q);
            // (lanes of groups that come before; every other lane where a group has two)
            const int better = per_group == 1 ? larger_keys<G, 1>(mine) : 2 * larger_keys<G, 2>(mine);
            dropped = better >= g.groups_kept * per_group;
            if (!by_logit)
                sure = apart(live && !dropped ? v : INFINITY, live && dropped ? v : -INFINITY,
                             live ? fmaxf(fabsf(a), fabsf(a2)) : 0.f);
#pragma unroll
            for (int i = 0; i < KM; ++i) list[i] = dropped ? key_of(kOut, 255) : list[i];
        }
        merge_partner<0, KM>(list);
        merge_partner<1, KM>(list);
        if constexpr (G >= 8) merge_partner<2, KM>(list);
        if constexpr (G >= 16) merge_partner<3, KM>(list);
        // list: the token's KM largest, in every lane
        if (!by_logit) {
            // (the list falls: its ends bound |c|, and if the last is above minus infinity all are)
            const float first = key_value(list[0]);
            float last = first, gap = INFINITY;
#pragma unroll
            for (int j = 1; j < KM; ++j) {
                if (j < k) {
                    const float v = key_value(list[j]);
                    gap = fminf(gap, last - v);
                    last = v;
                }
            }
            const float tol = s_error + 0x1p-22f * fmaxf(fabsf(first), fabsf(last));
            // no others within the error of the last (of those that are out c is minus infinity)
            int near = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) near += !(c[i] < last - tol) ? 1 : 0;
            near = reduce<G>(dropped ? 0 : near, Add());
            sure = sure && last > -INFINITY && gap > tol && near <= k;
        }
        // gates: lane j has slots j, j + G, ..
        constexpr int SLOTS = KM > G ? KM / G : 1;
        float chosen[SLOTS];
        int id[SLOTS];
        float total = 0.f;
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            double mine = list[0];
#pragma unroll
            for (int j = 1; j < KM; ++j) mine = s_lane + u * G == j ? list[j] : mine;
            id[u] = key_index(mine);
            chosen[u] = 0.f;
            if (s_lane + u * G < k) {
                const float l = from[min(id[u], E - 1)];
                if (g.score == MOE_SCORE_SOFTMAX) chosen[u] = expf(l - (top == -INFINITY ? 0.f : top)) * inv;
                else chosen[u] = 1.f / (1.f + expf(-l));
            }
            total += chosen[u];
        }
        total = reduce<G>(total, Add());
        // Scores chosen by a bias may be denormals or zeros in 32 bits, their shares are not:
        // such a token's gates are made in 64 bits, with its choice.  (Not masked rows,
        // whose scores are zeros in 64 bits, too: a softmax of minus infinities, and sigmoids
        // of which the largest logit, the list's first where logits choose, is too low.)
        sure = sure && !(g.renormalise && total < 0x1p-26f && inv != 0.f &&
                         !(by_logit && key_value(list[0]) < kLeastLogit));
        if (has && sure) {
#pragma unroll
            for (int u = 0; u < SLOTS; ++u) {
                const int j = s_lane + u * G;
                if (j >= k) continue;
                ids[t * k + j] = id[u];
                const float v = g.renormalise ? (total == 0.f ? 0.f : chosen[u] / total) : chosen[u];
                gates[t * k + j] = g.scale * v;
            }
        }
        const uint64_t unsure = __ballot(has && !sure && s_lane == 0);
        if (lane == 0) s_again[wave][round] = unsure;
    }
    if (partial != nullptr) {
        // over the wave's tokens, then over the waves
        float* const w_sum = reinterpret_cast<float*>(s_buf);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            float v = sum[i];
#pragma unroll
            for (int off = G; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
            if (row == 0) w_sum[wave * EMAX + e0 + i] = v;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += 256)
            partial[static_cast<int64_t>(blockIdx.x) * E + e] =
                (w_sum[e] + w_sum[EMAX + e]) + (w_sum[2 * EMAX + e] + w_sum[3 * EMAX + e]);
        __syncthreads();
    }
    // the tokens whose choice is not certain, again (here, where no registers are held)
    wave_lds();
    for (int r = 0; r < round; ++r) {
        uint64_t again = s_again[wave][r];
        while (again != 0) {
            const int at = __builtin_ctzll(again);
            again &= again - 1;
            double unused[kEpl];
            choose64(g, logits, bias, first + r * step + at / G, s_buf[wave], ids, gates, unused);
        }
    }
}

// sums[e] = the sum of the blocks' partial sums, in a fixed order: 8 experts per
// workgroup, 128 threads each, so that up to 1024 blocks' are one load per lane in
// flight eight times.
__global__ __launch_bounds__(1024) void score_sums_kernel(const float* __restrict__ partial, int64_t blocks, int E,
                                                         float* __restrict__ sums) {
    __shared__ double s[16][8];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
    const int e = blockIdx.x * 8 + x;
    double v = 0;
    if (e < E) {
#pragma unroll 8
        for (int64_t b = y; b < blocks; b += 128) v += partial[b * E + e];
    }
#pragma unroll
    for (int off = 8; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
    if ((threadIdx.x & 63) < 8) s[threadIdx.x >> 6][x] = v;
    __syncthreads();
    if (threadIdx.x < 8 && e < E) {
        v = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += s[i][x];
        sums[e] = static_cast<float>(v);
    }
}

// ---- the gradient ------------------------------------------------------------------------
//
// With r_j = s_j / S (S the sum of the chosen s) slot j's share of s ds is
//   renormalised  u_j = scale r_j (dg_j - sum_i r_i dg_i)      otherwise  scale s_j dg_j
// and with ds = dscore_sums
//   sigmoid  dl_e = (u_e + s_e ds_e) (1 - s_e)
//   softmax  dl_e = u_e + s_e (ds_e - sum_i s_i ds_i - sum_j u_j)
// (s_j / S is one quotient: 1 / S may overflow; renormalised, the u_j add up to zero).
// A bias may choose experts of scores that are denormals or zeros in 32 bits.  Their r_j are
// taken of exp(l_j - m), m the largest chosen logit rounded up to a whole number (l_j - m is
// exact for l_j <= m <= 0; a sigmoid's 1 - s rounds to 1 here), and are 0 where the gates
// are: sigmoid scores of logits below kLeastLogit.
//
// G lanes per token, 8 experts each; lane j takes slots j, j + G, .. and leaves u in LDS
// under its expert.  Bound by the logits read and the gradients written: whole 16-byte
// words, two tokens of 256 experts in flight per wave (32768 x 256: 18 us, 3.8 TB/s; one token
// per wave in 4-byte words 42 us).  Without dscore_sums all but the
// chosen experts' gradients are zero (softmax: if renormalised), and only their logits
// are read.
template <int G, typename T, typename F>
__device__ __forceinline__ T reduce_wide(T v, F op) {
    v = reduce<(G < 16 ? G : 16)>(v, op);
    if constexpr (G >= 32) v = op(v, __shfl_xor(v, 16, 64));
    return v;
}

// s and 1 - s of a logit, neither by a difference.
__device__ __forceinline__ void sigmoid_parts(float l, float& s, float& rest) {
    const float x = expf(-fabsf(l)), p = __builtin_amdgcn_rcpf(1.f + x);
    s = l >= 0.f ? p : x * p;
    rest = l >= 0.f ? x * p : p;
    if (!(l == l)) s = rest = l;
}

template <int G, bool VEC, typename O>
__global__ __launch_bounds__(256) void route_scored_backward_kernel(moe_gating_t g, const float* __restrict__ logits,
                                                                   const int32_t* __restrict__ ids,
                                                                   const float* __restrict__ dgates,
                                                                   const float* __restrict__ dsums,
                                                                   O* __restrict__ dlogits) {
    constexpr int N = 8, TPW = 64 / G;
    __shared__ __attribute__((aligned(16))) float s_u[4][TPW * G * N];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane / G, s_lane = lane % G;
    const int E = g.E, k = g.k;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * TPW;
    if (t0 >= g.T) return;
    const bool has = t0 + row < g.T;
    const int64_t t = has ? t0 + row : g.T - 1;
    const bool softmax = g.score == MOE_SCORE_SOFTMAX;
    const bool sparse = dsums == nullptr && (!softmax || g.renormalise);
    const float* const from = logits + t * E;
    float* const u_of = s_u[wave] + row * G * N;
    // expert i of the lane
    auto expert = [&](int i) { return VEC ? 4 * (s_lane + G * (i / 4)) + i % 4 : s_lane + G * i; };
    float l[N], ds[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        l[i] = -INFINITY;
        ds[i] = 0.f;
    }
    if (!sparse) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                if (expert(i) < E) {
                    const float4 v = *reinterpret_cast<const float4*>(from + expert(i));
                    l[i] = v.x;
                    l[i + 1] = v.y;
                    l[i + 2] = v.z;
                    l[i + 3] = v.w;
                }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (expert(i) < E) l[i] = from[expert(i)];
        }
        if (dsums != nullptr) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (expert(i) < E) ds[i] = dsums[expert(i)];
        }
    }
    // the slots: up to MOE_MAX_TOPK / G of them per lane
    constexpr int SLOTS = (MOE_MAX_TOPK + G - 1) / G;
    int id[SLOTS];
    float dg[SLOTS], lc[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        const int at = s_lane + G * j;
        id[j] = at < k ? ids[t * k + at] : -1;
        if (id[j] >= E) id[j] = -1;
        dg[j] = at < k ? g.scale * dgates[t * k + at] : 0.f;
        lc[j] = id[j] >= 0 ? from[id[j]] : -INFINITY;
    }
    // whether an expert is in two slots of a token: it keeps one slot's number
    bool twice = false;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
        if (G * j < k && id[j] >= 0) u_of[id[j]] = static_cast<float>(s_lane + G * j);
    wave_lds();
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
        if (G * j < k && id[j] >= 0) twice |= u_of[id[j]] != static_cast<float>(s_lane + G * j);
    wave_lds();
#pragma unroll
    for (int i = 0; i < N; ++i) u_of[s_lane + G * i] = 0.f;
    // scores
    float top = -INFINITY, inv = 0.f;
    float s[N], rest[N];
    if (softmax) {
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, l[i]);
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) top = fmaxf(top, lc[j]);
        top = reduce_wide<G>(top, Max());
        if (top == -INFINITY) top = 0.f;
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = expf(l[i] - top);
            z += s[i];
        }
        z = reduce_wide<G>(z, Add());
        // (sparse: the chosen experts' shares do not depend on it)
        inv = sparse ? 1.f : (z == 0.f ? 0.f : 1.f / z);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] *= inv;
            rest[i] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            sigmoid_parts(l[i], s[i], rest[i]);
            if (sparse) s[i] = 0.f;
        }
    }
    float sc[SLOTS], u[SLOTS], restc[SLOTS], total = 0.f, mean = 0.f, all = 0.f;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        restc[j] = 1.f;
        if (softmax) sc[j] = expf(lc[j] - top) * inv;
        else sigmoid_parts(lc[j], sc[j], restc[j]);
        if (id[j] < 0) sc[j] = 0.f;
        total += sc[j];
    }
    if (g.renormalise) {
        total = reduce_wide<G>(total, Add());
        const bool small = total < 0x1p-26f;
        if (__builtin_expect(__ballot(small) != 0, 0)) {
            float most = -INFINITY, w[SLOTS], sum = 0.f;
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) most = fmaxf(most, lc[j]);
            most = reduce_wide<G>(most, Max());
            const bool none = softmax ? most == -INFINITY : most < kLeastLogit;
            most = ceilf(most);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                w[j] = id[j] < 0 || none ? 0.f : expf(lc[j] - most);
                sum += w[j];
            }
            sum = reduce_wide<G>(sum, Add());
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) sc[j] = small ? w[j] : sc[j];
            total = small ? sum : total;
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            sc[j] = total == 0.f ? 0.f : sc[j] / total;
            mean += sc[j] * dg[j];
        }
        mean = reduce_wide<G>(mean, Add());
    }
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        u[j] = sc[j] * (dg[j] - mean);
        if (!g.renormalise) all += u[j];
    }
    wave_lds();
    if (__builtin_expect(__ballot(twice) == 0, 1)) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
            if (id[j] >= 0) u_of[id[j]] = sparse ? u[j] * restc[j] : u[j];
    } else {
        // (not what a routing gives: one slot after the other, for sums in their order)
        for (int q = 0; q < k; ++q) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
                if (s_lane + G * j == q && id[j] >= 0) u_of[id[j]] += sparse ? u[j] * restc[j] : u[j];
            wave_lds();
        }
    }
    if (softmax) {
#pragma unroll
        for (int i = 0; i < N; ++i) all += s[i] * ds[i];
        all = reduce_wide<G>(all, Add());
    }
    wave_lds();
    if (!has) return;
    O* const out = dlogits + t * E;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float ue = u_of[VEC ? 4 * (s_lane + G * (i / 4)) + i % 4 : s_lane + G * i];
        v[i] = sparse ? ue : (softmax ? ue + s[i] * (ds[i] - all) : (ue + s[i] * ds[i]) * rest[i]);
    }
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            if (expert(i) >= E) continue;
            if constexpr (sizeof(O) == 4)
                *reinterpret_cast<float4*>(out + expert(i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            else
                *reinterpret_cast<uint2*>(out + expert(i)) = make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (expert(i) < E) out[expert(i)] = static_cast<O>(v[i]);
    }
}

}  // namespace

// Workgroups: one round of tokens each up to 1024 of them, then up to kMaxRounds
// (each lane adds that many scores in 32 bits).
int64_t route_scored_blocks(const moe_gating_t& g) {
    const int64_t per_round = 4 * (64 / route_kernel(g).lanes);
    const int64_t rounds = ceil_div(g.T, per_round);
    return std::max(std::min<int64_t>(rounds, 1024), ceil_div(rounds, kMaxRounds));
}

hipError_t launch_route_scored(const moe_gating_t& g, const float* logits, const float* bias, int32_t* ids,
                               float* gates, float* score_sums, float* partial, hipStream_t s) {
    const int64_t blocks = route_scored_blocks(g);
    float* const sums = score_sums != nullptr ? partial : nullptr;
    if (blocks > 0) {
        const unsigned grid = static_cast<unsigned>(blocks);
        const RouteKernel kernel = route_kernel(g);
#define MOE_ROUTE_LIST(G, EPL, VEC, KM) route_scored_kernel<G, EPL, VEC, KM><<<grid, 256, 0, s>>>(g, logits, bias, ids, gates, sums)
#define MOE_ROUTE_K(G, EPL, VEC)                                        \
    do {                                                                \
        if (kernel.list == 4) MOE_ROUTE_LIST(G, EPL, VEC, 4);           \
        else if (kernel.list == 8) MOE_ROUTE_LIST(G, EPL, VEC, 8);      \
        else MOE_ROUTE_LIST(G, EPL, VEC, kMaxList);                     \
    } while (0)
#define MOE_ROUTE(G, EPL)                            \
    do {                                             \
        if (kernel.words) MOE_ROUTE_K(G, EPL, true); \
        else MOE_ROUTE_K(G, EPL, false);             \
    } while (0)
        if (kernel.list == 0) route_scored_wave_kernel<<<grid, 256, 0, s>>>(g, logits, bias, ids, gates, sums);
        else if (kernel.lanes == 4) MOE_ROUTE(4, 8);
        else if (kernel.lanes == 8) MOE_ROUTE(8, 8);
        else if (kernel.per_lane == 8) MOE_ROUTE(16, 8);
        else MOE_ROUTE(16, 16);
#undef MOE_ROUTE
#undef MOE_ROUTE_K
#undef MOE_ROUTE_LIST
    }
    if (score_sums != nullptr)
        score_sums_kernel<<<static_cast<unsigned>(ceil_div(g.E, 8)), 1024, 0, s>>>(partial, blocks, g.E, score_sums);
    return hipGetLastError();
}

namespace {

template <typename O>
void start_backward(const moe_gating_t& g, const float* logits, const int32_t* ids, const float* dgates,
                    const float* dsums, O* dlogits, hipStream_t s) {
    const RouteBackKernel kernel = route_back_kernel(g);
    const unsigned grid = static_cast<unsigned>(ceil_div(g.T, 4 * (64 / kernel.lanes)));
#define MOE_BACK(G)                                                                                              \
    do {                                                                                                         \
        if (kernel.words) route_scored_backward_kernel<G, true><<<grid, 256, 0, s>>>(g, logits, ids, dgates, dsums, dlogits); \
        else route_scored_backward_kernel<G, false><<<grid, 256, 0, s>>>(g, logits, ids, dgates, dsums, dlogits);    \
    } while (0)
    switch (kernel.lanes) {
        case 4: MOE_BACK(4); break;
        case 8: MOE_BACK(8); break;
        case 16: MOE_BACK(16); break;
        default: MOE_BACK(32); break;
    }
#undef MOE_BACK
}

}  // namespace

hipError_t launch_route_scored_backward(const moe_gating_t& g, const float* logits, const int32_t* ids,
                                        const float* dgates, const float* dscore_sums, int dtype, void* dlogits,
                                        hipStream_t s) {
    if (dtype == MOE_DTYPE_BF16)
        start_backward(g, logits, ids, dgates, dscore_sums, static_cast<__bf16*>(dlogits), s);
    else
        start_backward(g, logits, ids, dgates, dscore_sums, static_cast<float*>(dlogits), s);
    return hipGetLastError();
}

}  // namespace moe
