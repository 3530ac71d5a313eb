// The router by scores, and the gradient of its gates.
//
//   s = sigmoid(l) or softmax(l);  c = s + bias (no bias: the order of l);
//   groups_kept of the groups by their best choice or the sum of their two
//   best; the k best of these; gate = scale * s [/ sum of the chosen s]
//
// Which experts are chosen is a whole number, so it has to be right where two
// choices are nearer than fp32 tells apart: the fp32 values decide when every
// difference that matters exceeds both values' error, and else the token is
// done again in 64 bits (route_exact).  Without a bias the experts' order is
// the logits' own and needs no such care; the groups' does when two scores are
// added.
//
// Warp kernel: one warp per token, the choices in shared memory.  k rounds of
// a scan and two warp reductions; a further round looks at the best one left
// out.
#include <float.h>

#include "block_ops.cuh"
#include "expert_common.cuh"
#include "route_select.cuh"
#include "row_math.cuh"

namespace a2av {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kWarps = 4;  // warps per block, each on its own tokens

// A logit as the rule reads it: NaN the lowest finite value, infinities the ends, -0 as +0.
__device__ __forceinline__ float clean_logit(float v) { return fminf(fmaxf(v, -FLT_MAX), FLT_MAX) + 0.0f; }
// A choice: NaN as -infinity, -0 as +0.
__device__ __forceinline__ float clean_choice(float c) { return fmaxf(c, -INFINITY) + 0.0f; }

// 1 / (1 + exp(-l)) with the fast exponential and reciprocal: the exponential is off by 2 units of 2^-23 and by its
// argument's rounding, 1.5 * |l| * 2^-24, which the factor 1 - s damps; the sum and the reciprocal add 3 * 2^-24: below
// 2^-21 of s.
__device__ __forceinline__ float fast_sigmoid(float l) { return __fdividef(1.0f, 1.0f + __expf(-l)); }

// Bound of the error of an fp32 choice of size |c|.  Sigmoid: fast_sigmoid's, and the bias' addition.  Softmax: every
// score is at most `top`; exponential, sum (at most 32 terms in a row, then a tree) and quotient are off by less than
// 64 * 2^-24 of it together.
__device__ __forceinline__ float error_of(bool sigmoid, float top, float c) {
    return (sigmoid ? 0x1p-21f : top * 0x1p-18f) + fabsf(c) * 0x1p-23f;
}
// Whether choice c may in truth lie above `last`, which fp32 puts ahead of it.  Two infinite ones are equal as they stand.
__device__ __forceinline__ bool too_near(bool sigmoid, float top, float last, float c) {
    return !(last - c >= error_of(sigmoid, top, last) + error_of(sigmoid, top, c)) && !(last == c && isinf(c));
}

__device__ __forceinline__ double exact_score(bool sigmoid, float l, float m, double z) {
    return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) / z;
}

// The token with logits `l`, chosen in 64 bits by a whole warp; `key` holds E doubles.  Lane j < k gets slot j's id.
__device__ __noinline__ int route_exact(const ScoreArgs &a, const float *l, double *key, int lane) {
    const int E = a.g.E, k = a.g.k, size = E / a.groups;
    float m = -FLT_MAX;
    double z = 1.0;
    if (!a.sigmoid) {
        for (int e = lane; e < E; e += 32) m = fmaxf(m, clean_logit(__ldg(l + e)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        z = 0.0;
        for (int e = lane; e < E; e += 32) z += exp((double)clean_logit(__ldg(l + e)) - (double)m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    }
    for (int e = lane; e < E; e += 32) {
        const float v = clean_logit(__ldg(l + e));
        key[e] = a.bias ? fmax(exact_score(a.sigmoid, v, m, z) + (double)__ldg(a.bias + e), -(double)INFINITY) : (double)v;
    }
    __syncwarp();
    uint64_t keep = ~0ull;
    if (a.kept < a.groups) {
        double value[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int gi = q * 32 + lane;
            double b1 = -INFINITY, b2 = -INFINITY;
            if (gi < a.groups)
                for (int e = gi * size; e < (gi + 1) * size; ++e) {
                    const double c = key[e];
                    b2 = fmax(b2, fmin(b1, c));
                    b1 = fmax(b1, c);
                }
            value[q] = a.best == 1 ? b1
                       : a.bias    ? fmax(b1 + b2, -(double)INFINITY)
                                   : exact_score(a.sigmoid, (float)b1, m, z) + exact_score(a.sigmoid, (float)b2, m, z);
        }
        int before[2] = {0, 0};
        for (int gi = 0; gi < a.groups; ++gi) {
            const double v = __shfl_sync(kAll, gi < 32 ? value[0] : value[1], gi & 31);
#pragma unroll
            for (int q = 0; q < 2; ++q) before[q] += v > value[q] || (v == value[q] && gi < q * 32 + lane);
        }
        keep = (uint64_t)__ballot_sync(kAll, before[0] < a.kept && lane < a.groups) |
               (uint64_t)__ballot_sync(kAll, before[1] < a.kept && lane + 32 < a.groups) << 32;
    }
    int mine = -1;
    for (int j = 0; j < k; ++j) {
        double best = -INFINITY;
        int id = E;
        for (int e = lane; e < E; e += 32) {
            const double c = key[e];  // NaN: taken
            if ((keep >> (e / size) & 1) && (c > best || (c == best && id == E))) {
                best = c;
                id = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double c = __shfl_xor_sync(kAll, best, o);
            const int i = __shfl_xor_sync(kAll, id, o);
            if (i < E && (id == E || c > best || (c == best && i < id))) {
                best = c;
                id = i;
            }
        }
        if (lane == (id & 31)) key[id] = NAN;
        __syncwarp();
        if (lane == j) mine = id;
    }
    return mine;
}

// The gate of the slot in lane j < k, from its cleaned logit; m and z are the softmax's maximum and sum.
__device__ __forceinline__ float chosen_gate(const ScoreArgs &a, float l, bool in, float m, float z) {
    if (a.renorm) {
        // sigmoid: exp(min(l, 0)) / (1 + exp(-|l|)), over a common exp(M), so that it cannot vanish for every slot
        const float base = a.sigmoid ? fminf(l, 0.0f) : l;
        float top = in ? base : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        float e = in ? expf(base - top) : 0.0f;
        if (a.sigmoid) e = __fdiv_rn(e, 1.0f + expf(-fabsf(l)));
        return a.scale * __fdiv_rn(e, warp_sum(e));
    }
    if (!a.sigmoid) return a.scale * __fdiv_rn(expf(l - m), z);
    const float e = expf(-fabsf(l));
    return a.scale * __fdiv_rn(l >= 0.0f ? 1.0f : e, 1.0f + e);
}

// A group's value out of its best choices (without a bias they are logits), and a bound of its error.  A sum that
// overflows, or one of two infinities, is left to the 64-bit form.
__device__ __forceinline__ void group_value(const ScoreArgs &a, float b1, float b2, float m, float top, float &value,
                                            float &off) {
    if (a.best == 1) {
        value = b1;
        off = a.bias && !isinf(b1) ? error_of(a.sigmoid, top, b1) : 0.0f;
        return;
    }
    if (!a.bias) {  // the softmax's are not divided by their sum
        b1 = a.sigmoid ? fast_sigmoid(b1) : __expf(b1 - m);
        b2 = a.sigmoid ? fast_sigmoid(b2) : __expf(b2 - m);
        top = 1.0f;
    }
    value = clean_choice(b1 + b2);
    off = value == -INFINITY && b1 < INFINITY && b2 == -INFINITY ? 0.0f
          : isinf(b1) || isinf(b2) || isinf(value)               ? INFINITY
                                                   : error_of(a.sigmoid, top, b1) + error_of(a.sigmoid, top, b2) +
                                                         fabsf(value) * 0x1p-23f;
}

// One token by a warp: the fp32 choice, `room` E doubles.
__device__ __forceinline__ void route_one(const ScoreArgs &a, long long u, double *room, int lane) {
    const int E = a.g.E, k = a.g.k, size = E / a.groups;
    const float *l = a.logits + (size_t)u * E;
    uint32_t *key = reinterpret_cast<uint32_t *>(room);
    float m = -FLT_MAX, z = 0.0f;
    if (!a.sigmoid) {
        for (int e = lane; e < E; e += 32) m = fmaxf(m, clean_logit(__ldg(l + e)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (a.bias || !a.renorm) {
            float part = 0.0f;
            int n = 0;
            for (int e = lane; e < E; e += 32) {
                part += __expf(clean_logit(__ldg(l + e)) - m);
                if (++n % 32 == 0) {  // at most 32 terms in a row
                    z += part;
                    part = 0.0f;
                }
            }
            z = warp_sum(z + part);
        }
    }
    const float top = a.sigmoid ? 1.0f : __fdividef(1.0f, z);
    for (int e = lane; e < E; e += 32) {
        const float v = clean_logit(__ldg(l + e));
        float c = v;
        if (a.bias) c = clean_choice((a.sigmoid ? fast_sigmoid(v) : __expf(v - m) * top) + __ldg(a.bias + e));
        key[e] = order_key(c);
    }
    __syncwarp();
    bool near = false;
    if (a.kept < a.groups) {
        // a group's value, and the error it may have
        float value[2], off[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int gi = q * 32 + lane;
            uint32_t b1 = 0, b2 = 0;
            value[q] = -INFINITY;
            off[q] = 0.0f;
            if (gi >= a.groups) continue;
            for (int e = gi * size; e < (gi + 1) * size; ++e) {
                const uint32_t c = key[e];
                b2 = max(b2, min(b1, c));
                b1 = max(b1, c);
            }
            group_value(a, order_value(b1), a.best == 2 ? order_value(b2) : 0.0f, m, top, value[q], off[q]);
        }
        int before[2] = {0, 0};
        for (int gi = 0; gi < a.groups; ++gi) {
            const float v = __shfl_sync(kAll, gi < 32 ? value[0] : value[1], gi & 31);
#pragma unroll
            for (int q = 0; q < 2; ++q) before[q] += v > value[q] || (v == value[q] && gi < q * 32 + lane);
        }
        const bool in[2] = {before[0] < a.kept && lane < a.groups, before[1] < a.kept && lane + 32 < a.groups};
        const uint64_t keep = (uint64_t)__ballot_sync(kAll, in[0]) | (uint64_t)__ballot_sync(kAll, in[1]) << 32;
        if (a.bias || a.best == 2) {
            // the least that a kept one may be and the most that another may
            float lo = INFINITY, hi = -INFINITY;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (q * 32 + lane < a.groups) {
                    if (in[q]) lo = fminf(lo, value[q] - off[q]);
                    else hi = fmaxf(hi, value[q] + off[q]);
                }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(kAll, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, o));
            }
            near = !(lo >= hi);
        }
        for (int e = lane; e < E; e += 32)
            if (!(keep >> (e / size) & 1)) key[e] = 0u;
        __syncwarp();
    }
    int mine = -1;
    float last = 0.0f;
    for (int j = 0; j < k + (a.bias ? 1 : 0) && !near; ++j) {
        uint32_t best = 0u;
        int id = E;
        for (int e = lane; e < E; e += 32)
            if (key[e] > best) {
                best = key[e];
                id = e;
            }
        const uint32_t most = __reduce_max_sync(kAll, best);
        if (most == 0u) break;  // k of the kept groups' experts are all there are
        id = (int)__reduce_min_sync(kAll, best == most ? (uint32_t)id : 0xffffffffu);
        const float c = order_value(most);
        if (a.bias && j > 0) near = too_near(a.sigmoid, top, last, c);
        last = c;
        if (j == k) break;
        if (lane == (id & 31)) key[id] = 0u;
        __syncwarp();
        if (lane == j) mine = id;
    }
    __syncwarp();
    if (near) mine = route_exact(a, l, room, lane);
    const bool in = lane < k;
    const float g = chosen_gate(a, in ? clean_logit(__ldg(l + mine)) : 0.0f, in, m, z);
    if (in) {
        a.idx[(size_t)u * k + lane] = mine;
        a.gate[(size_t)u * k + lane] = g;
    }
    __syncwarp();
}

__device__ __forceinline__ bool token_active(const int32_t *num_tokens, int T, int u) {
    if (!num_tokens) return true;
    const int s = u / T;
    return u - s * T < active_tokens(num_tokens, s, T);
}

__global__ void __launch_bounds__(32 * kWarps) route_scores_kernel(const ScoreArgs a) {
    extern __shared__ __align__(16) unsigned char sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double *room = reinterpret_cast<double *>(sm) + (size_t)warp * a.g.E;
    const int ntok = a.g.R * a.g.T;
    grid_dependency_wait();
    for (long long u = (long long)blockIdx.x * kWarps + warp; u < ntok; u += (long long)gridDim.x * kWarps)
        if (token_active(a.num_tokens, a.g.T, (int)u)) route_one(a, u, room, lane);
}

// The gradient.  One warp per token: lane j takes slot j, its value goes to the id's place in a row in shared memory
// that is zero otherwise, and the row is stored.  With the whole softmax every place gets -p * sum, too.
//   renormalised softmax r:   scale * r_j * (d_j - sum d r)
//   renormalised sigmoid:     the same times 1 - s_j
//   sigmoid:                  scale * d_j * s_j * (1 - s_j)
//   softmax:                  scale * (p_j d_j - p * sum p d)
__global__ void __launch_bounds__(32 * kWarps) route_scores_grad_kernel(const ScoreArgs a) {
    extern __shared__ __align__(16) unsigned char sm[];
    const int E = a.g.E, k = a.g.k, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *row = reinterpret_cast<float *>(sm) + (size_t)warp * E;
    for (int e = lane; e < E; e += 32) row[e] = 0.0f;
    __syncwarp();
    grid_dependency_wait();
    const int ntok = a.g.R * a.g.T;
    const bool dense = !a.sigmoid && !a.renorm;
    for (long long u = (long long)blockIdx.x * kWarps + warp; u < ntok; u += (long long)gridDim.x * kWarps) {
        if (!token_active(a.num_tokens, a.g.T, (int)u)) continue;
        const float *l = a.logits + (size_t)u * E;
        const int id = lane < k ? __ldg(a.idx + (size_t)u * k + lane) : -1;
        const bool in = (uint32_t)id < (uint32_t)E;
        if (lane < k && !in) atomicOr(a.status, A2AV_DEV_BAD_EXPERT);
        const float d = in ? __ldg(a.d_gate + (size_t)u * k + lane) : 0.0f;
        const float v = in ? clean_logit(__ldg(l + id)) : 0.0f;
        const float ea = expf(-fabsf(v));
        const float rest = a.sigmoid ? __fdiv_rn(v >= 0.0f ? ea : 1.0f, 1.0f + ea) : 1.0f;  // 1 - s
        float m = -FLT_MAX, z = 1.0f, val;
        if (dense) {
            for (int e = lane; e < E; e += 32) m = fmaxf(m, clean_logit(__ldg(l + e)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
            z = 0.0f;
            for (int e = lane; e < E; e += 32) z += expf(clean_logit(__ldg(l + e)) - m);
            z = warp_sum(z);
            val = in ? a.scale * d * __fdiv_rn(expf(v - m), z) : 0.0f;
        } else if (a.renorm) {
            const float base = a.sigmoid ? fminf(v, 0.0f) : v;
            float top = in ? base : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
            float e = in ? expf(base - top) : 0.0f;
            if (a.sigmoid) e = __fdiv_rn(e, 1.0f + ea);
            const float sum = warp_sum(e), r = in ? __fdiv_rn(e, sum) : 0.0f, dot = warp_sum(r * d);
            val = in ? a.scale * r * (d - dot) * rest : 0.0f;
        } else {
            val = in ? a.scale * d * __fdiv_rn(v >= 0.0f ? 1.0f : ea, 1.0f + ea) * rest : 0.0f;
        }
        float all = 0.0f;  // an id that occurs twice: both slots' values, added in slot order by each
        for (int j = 0; j < k; ++j) {
            const int other = __shfl_sync(kAll, id, j);
            const float w = __shfl_sync(kAll, val, j);
            if (other == id) all += w;
        }
        const float sum = dense ? warp_sum(val) : 0.0f;
        if (in) row[id] = all;
        __syncwarp();
        float *out = a.d_logits + (size_t)u * E;
        for (int e = lane; e < E; e += 32)
            out[e] = dense ? row[e] - sum * __fdiv_rn(expf(clean_logit(__ldg(l + e)) - m), z) : row[e];
        __syncwarp();
        if (in) row[id] = 0.0f;
        __syncwarp();
    }
}

template <typename Kernel>
cudaError_t launch_tokens(Kernel kernel, std::atomic<uint64_t> &done, size_t per_expert, const a2av_plan_s &p,
                          const ScoreArgs &a, cudaStream_t s) {
    const cudaError_t e = allow_smem(kernel, done, p.cfg.device, kWarps * per_expert * kMaxExperts);
    if (e != cudaSuccess) return e;
    const size_t smem = kWarps * per_expert * (size_t)a.g.E;
    const long long want = ((long long)a.g.R * a.g.T + kWarps - 1) / kWarps;
    const long long fit = (long long)(200 * 1024 / (smem + 1024)), cap = (long long)p.num_sms * (fit < 12 ? fit : 12);
    return launch_pdl(kernel, (int)(want < cap ? want : cap), 32 * kWarps, smem, s, a);
}

}  // namespace

cudaError_t launch_route_scores(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    return launch_tokens(route_scores_kernel, done, sizeof(double), p, a, s);
}

cudaError_t launch_route_scores_grad(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    return launch_tokens(route_scores_grad_kernel, done, sizeof(float), p, a, s);
}

}  // namespace a2av
