// Routing by scores, with a balance bias and groups of experts, and its gradient.
//
//   s[t, e]  = sigmoid(l[t, e]), or softmax over the experts
//   c[t, e]  = s[t, e] + bias[e]             (the order of choice, not the gates)
//   group    value: the sum of its group_top largest c; the groups_kept best stay
//   ids      the k largest c of the groups that stay, ties to the lower expert
//   gates    scale * s of the chosen, over the sum of the chosen s if renormalised
//
// c decides between experts, so it is computed in 64 bits: two scores that
// differ in the 30th bit are in the right order.  Without a bias c has the order
// of the logits, which then stand for it (unless groups are valued by sums).
#include <limits.h>
#include <math.h>

#include "device_util.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kEpl = MOE_MAX_EXPERTS / 64;  // experts per lane: lane, lane + 64, ..

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmax(v, __shfl_xor(v, off, 64));
    return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Whether (v, e) is chosen before (w, f).
__device__ __forceinline__ bool before(double v, int e, double w, int f) { return v > w || (v == w && e < f); }

// One wave per token, kTokens tokens per wave one after the other.
constexpr int kTokens = 8;

__global__ __launch_bounds__(256) void route_scored_kernel(moe_gating_t g, const float* __restrict__ logits,
                                                          const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                          float* __restrict__ gates, float* __restrict__ partial) {
    __shared__ double s_c[4][MOE_MAX_EXPERTS];
    __shared__ double s_v[4][MOE_MAX_EXPERTS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E = g.E, k = g.k;
    const int size = E / g.groups;
    const bool limited = g.groups_kept < g.groups;
    const bool by_logit = bias == nullptr && (!limited || g.group_top == 1);
    double* const c_of = s_c[wave];
    double* const v_of = s_v[wave];
    double sum[kEpl] = {};
    for (int i = 0; i < kTokens; ++i) {
        const int64_t t = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * kTokens + i;
        if (t >= g.T) break;
        double l[kEpl], s[kEpl], c[kEpl];
        double top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            const int e = lane + 64 * j;
            l[j] = e < E ? logits[t * E + e] : -INFINITY;
            top = fmax(top, l[j]);
        }
        if (g.score == MOE_SCORE_SOFTMAX) {
            top = wave_max(top);
            double z = 0;
#pragma unroll
            for (int j = 0; j < kEpl; ++j) {
                // (a row of minus infinities: all scores zero)
                s[j] = top == -INFINITY ? 0 : exp(l[j] - top);
                z += lane + 64 * j < E ? s[j] : 0;
            }
            z = wave_sum(z);
#pragma unroll
            for (int j = 0; j < kEpl; ++j) s[j] = z == 0 ? 0 : s[j] / z;
        } else {
#pragma unroll
            for (int j = 0; j < kEpl; ++j) s[j] = 1.0 / (1.0 + exp(-l[j]));
        }
        bool live[kEpl];
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            const int e = lane + 64 * j;
            live[j] = e < E;
            c[j] = by_logit ? l[j] : s[j] + (bias != nullptr && e < E ? bias[e] : 0.f);
            if (!(c[j] == c[j])) c[j] = -INFINITY;  // (a NaN comes last)
            if (live[j]) sum[j] += s[j];
        }
        if (limited) {
#pragma unroll
            for (int j = 0; j < kEpl; ++j)
                if (live[j]) c_of[lane + 64 * j] = c[j];
            __builtin_amdgcn_wave_barrier();
            for (int q = lane; q < g.groups; q += 64) {
                double a = -INFINITY, b = -INFINITY;
                for (int e = q * size; e < (q + 1) * size; ++e) {
                    const double v = c_of[e];
                    b = fmax(b, fmin(a, v));
                    a = fmax(a, v);
                }
                const double v = g.group_top == 2 && size > 1 ? a + b : a;
                v_of[q] = v == v ? v : -INFINITY;
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < kEpl; ++j) {
                if (!live[j]) continue;
                const int mine = (lane + 64 * j) / size;
                int rank = 0;
                for (int q = 0; q < g.groups; ++q) rank += before(v_of[q], q, v_of[mine], mine) ? 1 : 0;
                live[j] = rank < g.groups_kept;
            }
        }
        double my_s = 0;
        int my_e = 0;
        for (int r = 0; r < k; ++r) {
            double bv = -INFINITY, bs = 0;
            int be = INT_MAX;
#pragma unroll
            for (int j = 0; j < kEpl; ++j) {
                const int e = lane + 64 * j;
                if (live[j] && (be == INT_MAX || before(c[j], e, bv, be))) {
                    bv = c[j];
                    be = e;
                    bs = s[j];
                }
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) {
                const double ov = __shfl_xor(bv, off, 64), os = __shfl_xor(bs, off, 64);
                const int oe = __shfl_xor(be, off, 64);
                if (oe != INT_MAX && (be == INT_MAX || before(ov, oe, bv, be))) {
                    bv = ov;
                    be = oe;
                    bs = os;
                }
            }
#pragma unroll
            for (int j = 0; j < kEpl; ++j)
                if (lane + 64 * j == be) live[j] = false;
            if (lane == r) {
                my_s = bs;
                my_e = be;
            }
        }
        const double total = wave_sum(my_s);
        if (lane < k) {
            ids[t * k + lane] = my_e;
            const double v = g.renormalise ? (total == 0 ? 0 : my_s / total) : my_s;
            gates[t * k + lane] = static_cast<float>(g.scale * v);
        }
        __builtin_amdgcn_wave_barrier();
    }
    if (partial == nullptr) return;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEpl; ++j) s_c[wave][lane + 64 * j] = sum[j];
    __syncthreads();
    const int e = threadIdx.x;
    if (e < E)
        partial[static_cast<int64_t>(blockIdx.x) * E + e] =
            static_cast<float>((s_c[0][e] + s_c[1][e]) + (s_c[2][e] + s_c[3][e]));
}

// sums[e] = the sum of the blocks' partial sums, in a fixed order.
__global__ __launch_bounds__(256) void score_sums_kernel(const float* __restrict__ partial, int64_t blocks, int E,
                                                        float* __restrict__ sums) {
    __shared__ double s[256];
    double v = 0;
    for (int64_t b = threadIdx.x; b < blocks; b += 256) v += partial[b * E + blockIdx.x];
    s[threadIdx.x] = v;
    __syncthreads();
    for (int off = 128; off > 0; off >>= 1) {
        if (threadIdx.x < off) s[threadIdx.x] += s[threadIdx.x + off];
        __syncthreads();
    }
    if (threadIdx.x == 0) sums[blockIdx.x] = static_cast<float>(s[0]);
}

// The gradient: with r_j = s_j / S (S the sum of the chosen s) the chosen expert
// j's score has the derivative
//   renormalised  scale (dg_j - sum_i r_i dg_i) / S       otherwise  scale dg_j
// and every score that of its sum; then
//   sigmoid  dl = ds s (1 - s)          softmax  dl = s (ds - sum_i s_i ds_i)
// where s_j / S is taken as one quotient (1 / S may overflow).  One wave per token.
template <typename O>
__global__ __launch_bounds__(256) void route_scored_backward_kernel(moe_gating_t g, const float* __restrict__ logits,
                                                                   const int32_t* __restrict__ ids,
                                                                   const float* __restrict__ dgates,
                                                                   const float* __restrict__ dsums,
                                                                   O* __restrict__ dlogits) {
    const int lane = threadIdx.x & 63;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (t >= g.T) return;
    const int E = g.E, k = g.k;
    float s[kEpl], rest[kEpl], l[kEpl], ds[kEpl], dg[kEpl];
    bool hit[kEpl];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
        const int e = lane + 64 * j;
        l[j] = e < E ? logits[t * E + e] : -INFINITY;
        top = fmaxf(top, l[j]);
        ds[j] = dsums != nullptr && e < E ? dsums[e] : 0.f;
        dg[j] = 0.f;
        hit[j] = false;
    }
    if (g.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            s[j] = top == -INFINITY || lane + 64 * j >= E ? 0.f : expf(l[j] - top);
            z += s[j];
        }
        z = wave_sum(z);
#pragma unroll
        for (int j = 0; j < kEpl; ++j) s[j] = z == 0.f ? 0.f : s[j] / z;
    } else {
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            s[j] = lane + 64 * j < E ? 1.f / (1.f + expf(-l[j])) : 0.f;
            rest[j] = 1.f / (1.f + expf(l[j]));
        }
    }
    for (int i = 0; i < k; ++i) {
        const int e = ids[t * k + i];
        const float v = g.scale * dgates[t * k + i];
#pragma unroll
        for (int j = 0; j < kEpl; ++j)
            if (lane + 64 * j == e) {
                dg[j] += v;
                hit[j] = true;
            }
    }
    // u: the chosen experts' share of s ds
    float u[kEpl], total = 0.f;
#pragma unroll
    for (int j = 0; j < kEpl; ++j) total += hit[j] ? s[j] : 0.f;
    if (g.renormalise) {
        total = wave_sum(total);
        float mean = 0.f;
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
            u[j] = hit[j] && total != 0.f ? s[j] / total : 0.f;
            mean += u[j] * dg[j];
        }
        mean = wave_sum(mean);
#pragma unroll
        for (int j = 0; j < kEpl; ++j) u[j] *= dg[j] - mean;
    } else {
#pragma unroll
        for (int j = 0; j < kEpl; ++j) u[j] = hit[j] ? s[j] * dg[j] : 0.f;
    }
    float mean = 0.f;
    if (g.score == MOE_SCORE_SOFTMAX) {
        // (renormalised, the chosen shares add up to zero)
#pragma unroll
        for (int j = 0; j < kEpl; ++j) mean += s[j] * ds[j] + (g.renormalise ? 0.f : u[j]);
        mean = wave_sum(mean);
    }
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
        const int e = lane + 64 * j;
        const float v = g.score == MOE_SCORE_SOFTMAX ? u[j] + s[j] * (ds[j] - mean) : (u[j] + s[j] * ds[j]) * rest[j];
        if (e < E) dlogits[t * E + e] = static_cast<O>(v);
    }
}

}  // namespace

int64_t route_scored_blocks(const moe_gating_t& g) { return ceil_div(g.T, 4 * kTokens); }

hipError_t launch_route_scored(const moe_gating_t& g, const float* logits, const float* bias, int32_t* ids,
                               float* gates, float* score_sums, float* partial, hipStream_t s) {
    const int64_t blocks = route_scored_blocks(g);
    if (blocks > 0)
        route_scored_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(g, logits, bias, ids, gates,
                                                                          score_sums != nullptr ? partial : nullptr);
    if (score_sums != nullptr) score_sums_kernel<<<static_cast<unsigned>(g.E), 256, 0, s>>>(partial, blocks, g.E, score_sums);
    return hipGetLastError();
}

hipError_t launch_route_scored_backward(const moe_gating_t& g, const float* logits, const int32_t* ids,
                                        const float* dgates, const float* dscore_sums, int dtype, void* dlogits,
                                        hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(ceil_div(g.T, 4));
    if (dtype == MOE_DTYPE_BF16)
        route_scored_backward_kernel<<<grid, 256, 0, s>>>(g, logits, ids, dgates, dscore_sums,
                                                          static_cast<__bf16*>(dlogits));
    else
        route_scored_backward_kernel<<<grid, 256, 0, s>>>(g, logits, ids, dgates, dscore_sums,
                                                          static_cast<float*>(dlogits));
    return hipGetLastError();
}

}  // namespace moe
