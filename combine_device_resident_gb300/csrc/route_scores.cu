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
// Warp kernel (any shape): one warp per token, the choices in shared memory.  k
// rounds of a scan and two warp reductions; a further round looks at the best
// one left out.  65,536 tokens of 512 logits, sigmoid with bias, top-8: 168 us (their 134 MB are 20): bound by the way
// through the rounds, each after the one before.  Lane kernel (E up to 256, k up to 8): four lanes per token, below.
#include <float.h>

#include <type_traits>

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

// exp(x) by the fast power of two, off by (2 + 1.17 |x|) * 2^-23 of itself; 0 below 2^-126.
__device__ __forceinline__ float fast_exp(float x) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
    return e;
}
// 1 / (1 + exp(-l)) with the fast exponential, whose error the factor 1 - s damps to
// (0.5 + 0.27) * 2^-23 at most, the sum's rounding, 2^-24, and the fast reciprocal's, 2^-23: below 2.3 * 2^-23.
__device__ __forceinline__ float fast_sigmoid(float l) {
    float s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + fast_exp(-l)));
    return s;
}

// Bound of the error of an fp32 choice of size |c|.  Sigmoid: fast_sigmoid's, and the bias' addition.  Softmax: every
// score is at most `top`; exponential, sum (at most 32 terms in a row, then a tree) and quotient are off by some 70 * 2^-24 of
// it at most, all but 5 of these by a factor common to the token's scores, so two such bounds (128 * 2^-24) hold a
// difference's error.
__device__ __forceinline__ float error_of(bool sigmoid, float top, float c) {
    return (sigmoid ? 2.4f * 0x1p-23f : top * 0x1p-18f) + fabsf(c) * 0x1p-24f;
}
// Whether choice c may in truth lie above `last`, which fp32 puts ahead of it.  Two infinite ones are equal as they stand.
__device__ __forceinline__ bool too_near(bool sigmoid, float top, float last, float c) {
    return !(last - c >= error_of(sigmoid, top, last) + error_of(sigmoid, top, c)) && !(last == c && isinf(c));
}

__device__ __forceinline__ double exact_score(bool sigmoid, float l, float m, double z) {
    return sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) / z;
}

// Order of doubles as that of signed integers (no NaN; -0 below +0, so add 0 first): the 64-bit pipe is slow here.
__device__ __forceinline__ long long order64(double v) {
    const long long b = __double_as_longlong(v + 0.0);
    return b ^ (b >> 63 & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double value64(long long k) {
    return __longlong_as_double(k ^ (k >> 63 & 0x7fffffffffffffffll));
}
constexpr long long kLow64 = -0x7fffffffffffffffll - 1;  // below every choice

// The token with logits `l`, chosen in 64 bits by a whole warp; `key` holds E words.  Lane j < k gets slot j's id.
__device__ __noinline__ int route_exact(const ScoreArgs &a, const float *l, long long *key, int lane) {
    const int E = a.g.E, k = a.g.k, size = E / a.groups;
    float m = -FLT_MAX;
    double z = 1.0;
    if (!a.sigmoid) {
        for (int e = lane; e < E; e += 32) m = fmaxf(m, clean_logit(__ldg(l + e)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        z = 0.0;
#pragma unroll 4
        for (int e = lane; e < E; e += 32) z += exp((double)clean_logit(__ldg(l + e)) - (double)m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    }
    if (a.bias) {
#pragma unroll 4
        for (int e = lane; e < E; e += 32)
            key[e] = order64(fmax(exact_score(a.sigmoid, clean_logit(__ldg(l + e)), m, z) + (double)__ldg(a.bias + e),
                                  -(double)INFINITY));
    } else {
        for (int e = lane; e < E; e += 32) key[e] = order64((double)clean_logit(__ldg(l + e)));
    }
    __syncwarp();
    uint64_t keep = ~0ull;
    if (a.kept < a.groups) {
        // lane gi and, from the 33rd group on, lane gi - 32 get group gi's two best
        long long first[2] = {kLow64, kLow64}, second[2] = {kLow64, kLow64};
        for (int gi = 0; gi < a.groups; ++gi) {
            long long b1 = kLow64, b2 = kLow64;
            for (int e = gi * size + lane; e < (gi + 1) * size; e += 32) {
                const long long c = key[e];
                b2 = max(b2, min(b1, c));
                b1 = max(b1, c);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const long long c1 = __shfl_xor_sync(kAll, b1, o), c2 = __shfl_xor_sync(kAll, b2, o);
                b2 = max(min(b1, c1), max(b2, c2));
                b1 = max(b1, c1);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (gi == q * 32 + lane) {
                    first[q] = b1;
                    second[q] = b2;
                }
        }
        long long value[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            value[q] = first[q];
            if (a.best == 2 && q * 32 + lane < a.groups) {
                const double b1 = value64(first[q]), b2 = value64(second[q]);
                value[q] = order64(a.bias ? fmax(b1 + b2, -(double)INFINITY)
                                          : exact_score(a.sigmoid, (float)b1, m, z) + exact_score(a.sigmoid, (float)b2, m, z));
            }
        }
        int before[2] = {0, 0};
        for (int gi = 0; gi < a.groups; ++gi) {
            const long long v = __shfl_sync(kAll, gi < 32 ? value[0] : value[1], gi & 31);
#pragma unroll
            for (int q = 0; q < 2; ++q) before[q] += v > value[q] || (v == value[q] && gi < q * 32 + lane);
        }
        keep = (uint64_t)__ballot_sync(kAll, before[0] < a.kept && lane < a.groups) |
               (uint64_t)__ballot_sync(kAll, before[1] < a.kept && lane + 32 < a.groups) << 32;
        for (int e = lane; e < E; e += 32)
            if (!(keep >> (e / size) & 1)) key[e] = kLow64;
        __syncwarp();
    }
    int mine = -1;
    for (int j = 0; j < k; ++j) {
        long long best = kLow64;
        int id = E;
        for (int e = lane; e < E; e += 32) {
            const long long c = key[e];
            if (c > best) {
                best = c;
                id = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const long long c = __shfl_xor_sync(kAll, best, o);
            const int i = __shfl_xor_sync(kAll, id, o);
            if (c > best || (c == best && i < id)) {
                best = c;
                id = i;
            }
        }
        if (lane == (id & 31)) key[id] = kLow64;
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

// A group's value out of its best choices (without a bias they are logits), and a bound of its error.  Of two best it is
// half the sum, which cannot overflow and has the sum's order.  An infinite choice is the bias, in 64 bits too, and so is
// one past 2^56, where no score moves it: the sum of two infinite ones, or of two equal ones that large, is exact.
__device__ __forceinline__ void group_value(const ScoreArgs &a, float b1, float b2, float m, float top, float &value,
                                            float &off) {
    if (a.best == 1) {
        value = b1;
        off = a.bias && !isinf(b1) ? error_of(a.sigmoid, top, b1) : 0.0f;
        return;
    }
    if (!a.bias) {  // the softmax's are not divided by their sum
        b1 = a.sigmoid ? fast_sigmoid(b1) : fast_exp(b1 - m);
        b2 = a.sigmoid ? fast_sigmoid(b2) : fast_exp(b2 - m);
        top = 1.0f;
    }
    value = clean_choice(fmaf(0.5f, b1, 0.5f * b2));
    off = 0.5f * (error_of(a.sigmoid, top, b1) + error_of(a.sigmoid, top, b2)) + fabsf(value) * 0x1p-23f;
    if (fmaxf(b1, -b2) > 0x1p56f && (b1 == b2 || isinf(b1) || isinf(b2))) off = 0.0f;
}

// One token by a warp: the fp32 choice, `room` E words of 64 bits.
__device__ __forceinline__ void route_one(const ScoreArgs &a, long long u, long long *room, int lane) {
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
                part += fast_exp(clean_logit(__ldg(l + e)) - m);
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
        if (a.bias) c = clean_choice((a.sigmoid ? fast_sigmoid(v) : fast_exp(v - m) * top) + __ldg(a.bias + e));
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
    long long *room = reinterpret_cast<long long *>(sm) + (size_t)warp * a.g.E;
    const int ntok = a.g.R * a.g.T;
    grid_dependency_wait();
    for (long long u = (long long)blockIdx.x * kWarps + warp; u < ntok; u += (long long)gridDim.x * kWarps)
        if (token_active(a.num_tokens, a.g.T, (int)u)) route_one(a, u, room, lane);
}

// ---- lane kernel ------------------------------------------------------------------
//
// Four lanes per token, eight tokens per warp.  Lane r of a token holds the 16-byte units r, r + 4, ... of its row in
// registers (NU of them), so every loop over logits is unrolled and none is read twice.  In order:
//   1. choices in place of logits; a copy of them in shared memory, for the few that are looked up by number later;
//   2. groups: lane r reads groups r, r + 4, ... out of the shared copy, each lane from another unit on (so that four lie on
//      different banks), and takes their two best; ranks by counting;
//   3. tau, a lower bound of the KMAX-th largest choice: the KMAX-th largest of maxima of disjoint sets (a lane's kept
//      units, by component);
//   4. the choices at or above tau (some ten of 256 for KMAX = 8) as bits, then as a list in shared memory;
//   5. each one's rank by counting those at or above it, a lane taking every fourth; ranks below k are the answer.
// A tie leaves a rank empty (of a slot, or behind the last one), and near neighbours are seen.  Then the warp ranks once more,
// equal choices by id, which is right where they come from equal logits and biases, and where at the border the first one
// behind them that does not is far enough; for the rest it orders the token's list in 64 bits (with a bias tau is lowered
// by the choices' errors, so that the list holds whatever may lie at the border).  Groups that are too near are settled
// in 64 bits before tau (keep_exact).  A list that is too long: route_one.
constexpr int kList = 32;  // candidates of a token
constexpr int kRanks = 16;  // room for a token's ranks, and for its groups' values
constexpr int kLaneGroups = 16;

template <int KMAX>
constexpr int tau_values() {  // that a lane gives to the bound
    return KMAX >= 4 ? KMAX / 2 : 1;
}

__device__ __forceinline__ void order2(float &a, float &b) {
    const float hi = fmaxf(a, b), lo = fminf(a, b);
    a = hi;
    b = lo;
}
__device__ __forceinline__ void sort4(float (&v)[4]) {
    order2(v[0], v[1]);
    order2(v[2], v[3]);
    order2(v[0], v[2]);
    order2(v[1], v[3]);
    order2(v[1], v[2]);
}
// The KMAX-th largest of what the token's four lanes give, sorted in descending order each.
template <int KMAX>
__device__ __forceinline__ float bound_of(const float (&g)[tau_values<KMAX>()]) {
    if constexpr (KMAX <= 2) {
        float a = g[0], b = __shfl_xor_sync(kAll, a, 1);
        order2(a, b);
        const float c = __shfl_xor_sync(kAll, a, 2), d = __shfl_xor_sync(kAll, b, 2);
        return KMAX == 1 ? fmaxf(a, c) : fmaxf(fminf(a, c), fmaxf(b, d));
    } else {
        constexpr int L = KMAX / 2;
        float c[KMAX];  // two lanes' values, mine and then the other's reversed: bitonic, to be sorted
#pragma unroll
        for (int i = 0; i < L; ++i) {
            c[i] = g[i];
            c[KMAX - 1 - i] = __shfl_xor_sync(kAll, g[i], 1);
        }
#pragma unroll
        for (int d = L; d >= 1; d >>= 1)
#pragma unroll
            for (int j = 0; j < KMAX; ++j)
                if ((j & d) == 0) order2(c[j], c[j + d]);
        float t = INFINITY;  // of two sorted lists of K, the K-th largest is min_i max(A_i, B_{K-1-i})
#pragma unroll
        for (int i = 0; i < KMAX; ++i) t = fminf(t, fmaxf(c[i], __shfl_xor_sync(kAll, c[KMAX - 1 - i], 2)));
        return t;
    }
}

// Row stride of the choices in shared memory, in 16-byte units: 4 mod 8, so that the eight lanes of two tokens lie on
// different banks.
__host__ __device__ constexpr int lane_stride(int E) { return (E / 4 + 7) / 8 * 8 + 4; }
struct LaneList {
    float key[8][kList + 4];  // candidates of the eight tokens, NaN behind them
    float best[8][kRanks];    // by rank; NaN where there is none
    alignas(4) uint8_t id[8][kList];
    uint8_t best_id[8][kRanks];
};
// A warp's share: the choices of eight tokens (also room for the warp kernel's token), the lists.
__host__ __device__ constexpr size_t lane_warp_bytes(int E) { return (size_t)8 * lane_stride(E) * 16 + sizeof(LaneList); }

__device__ __forceinline__ float &part_of(float4 &v, int c) { return c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w; }
// Two best of what two sides have.
__device__ __forceinline__ void merge2(float &a1, float &a2, float b1, float b2) {
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
}
__device__ __forceinline__ float token_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(kAll, v, 1));
    return fmaxf(v, __shfl_xor_sync(kAll, v, 2));
}
__device__ __forceinline__ float token_sum(float v) {
    v += __shfl_xor_sync(kAll, v, 1);
    return v + __shfl_xor_sync(kAll, v, 2);
}

// The n candidates of token u (its list's slot t), ordered in 64 bits by the whole warp.
__device__ __noinline__ void route_list(const ScoreArgs &a, int u, LaneList &list, int t, int n, int lane) {
    const float *l = a.logits + (size_t)u * a.g.E;
    const int id = lane < n ? list.id[t][lane] : 0;
    const float v = clean_logit(__ldg(l + id));
    float m = 0.0f, zf = 1.0f;
    double z = 1.0;
    if (!a.sigmoid && (a.bias || !a.renorm)) {
        m = -FLT_MAX;
        for (int e = lane; e < a.g.E; e += 32) m = fmaxf(m, clean_logit(__ldg(l + e)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        z = 0.0;
        for (int e = lane; e < a.g.E; e += 32) z += exp((double)clean_logit(__ldg(l + e)) - (double)m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
        zf = (float)z;
    }
    const long long c = order64(
        a.bias ? fmax(exact_score(a.sigmoid, v, m, z) + (double)__ldg(a.bias + id), -(double)INFINITY) : (double)v);
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const long long other = __shfl_sync(kAll, c, i);
        const int other_id = __shfl_sync(kAll, id, i);
        rank += other > c || (other == c && other_id < id);
    }
    if (lane < n && rank < a.g.k) list.best_id[t][rank] = id;
    __syncwarp();
    const bool in = lane < a.g.k;
    const int chosen = in ? list.best_id[t][lane] : 0;
    const float g = chosen_gate(a, in ? clean_logit(__ldg(l + chosen)) : 0.0f, in, m, zf);
    if (in) {
        a.idx[(size_t)u * a.g.k + lane] = chosen;
        a.gate[(size_t)u * a.g.k + lane] = g;
    }
    __syncwarp();
}

// The groups of token u (the warp's t-th) that are kept, as bits, its fp32 values left open.  floor[g]: choices of group g
// below it are none of its two best; `keys` the token's choices.  All ones where too many are not.
__device__ __noinline__ uint32_t keep_exact(const ScoreArgs &a, int u, const float *keys, const float *floor,
                                            uint8_t *ids, int lane) {
    const int E = a.g.E, size = E / a.groups;
    const float *l = a.logits + (size_t)u * E;
    int n = 0;
    for (int e = lane; e - lane < E; e += 32) {
        const bool in = e < E && keys[e] >= floor[e / size];
        const uint32_t all = __ballot_sync(kAll, in);
        const int pos = n + __popc(all & lanemask_lt());
        if (in && pos < kList) ids[pos] = (uint8_t)e;
        n += __popc(all);
    }
    __syncwarp();
    if (n > kList) return ~0u;
    float m = 0.0f;
    double z = 1.0;
    if (!a.sigmoid) {
        m = -FLT_MAX;
        for (int e = lane; e < E; e += 32) m = fmaxf(m, clean_logit(__ldg(l + e)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (a.bias) {  // else the scores' common divisor matters to no group
            z = 0.0;
#pragma unroll 4
            for (int e = lane; e < E; e += 32) z += exp((double)clean_logit(__ldg(l + e)) - (double)m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
        }
    }
    const int id = lane < n ? ids[lane] : 0;
    const float v = clean_logit(__ldg(l + id));
    const long long c = order64(
        a.bias ? fmax(exact_score(a.sigmoid, v, m, z) + (double)__ldg(a.bias + id), -(double)INFINITY) : (double)v);
    long long b1 = kLow64, b2 = kLow64;  // of group `lane`
    for (int i = 0; i < n; ++i) {
        const long long other = __shfl_sync(kAll, c, i);
        if (__shfl_sync(kAll, id, i) / size == lane) {
            b2 = max(b2, min(b1, other));
            b1 = max(b1, other);
        }
    }
    long long value = b1;
    if (a.best == 2 && lane < a.groups) {
        const double d1 = value64(b1), d2 = value64(b2);
        value = order64(a.bias ? fmax(d1 + d2, -(double)INFINITY)
                               : exact_score(a.sigmoid, (float)d1, m, z) + exact_score(a.sigmoid, (float)d2, m, z));
    }
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
        const long long other = __shfl_sync(kAll, value, g);
        before += other > value || (other == value && g < lane);
    }
    return __ballot_sync(kAll, lane < a.groups && before < a.kept);
}

// kFull: E is 16 * NU, so no unit is missing: taken for 128 and 256 experts without groups (65,536 tokens, sigmoid with
// bias, top-8: 21.6 us for 22.6 with the checks, and 33.6 for 35.1) and 256 in groups (39.2 for 46.8).  65,536 tokens of
// 256 logits, sigmoid with bias, 4 of 8 groups, top-8 take 39-42 us (their 71 MB are 10.5).  Bound by latency: some 2,300
// instructions a warp for eight tokens, a task's row asked for when the one before is done, half of the issue slots empty at 16 warps
// an SM; one warp per token takes 224.  Four blocks an SM with 128 registers: 35-38 us where five with 96 took 44 and three
// with 160 37 (with the groups merged in registers, which only groups of 16 and more allow).
template <int NU, int KMAX, bool kGroups, bool kFull>
__global__ void __launch_bounds__(32 * kWarps, 4) route_scores_lane_kernel(const ScoreArgs a) {
    extern __shared__ __align__(16) unsigned char sm[];
    constexpr int L = tau_values<KMAX>();
    const int E = a.g.E, k = a.g.k, nu = E / 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nwarps = blockDim.x >> 5, t = lane >> 2, r = lane & 3, stride = lane_stride(E);
    float4 *const bias4 = reinterpret_cast<float4 *>(sm);  // a NaN as -infinity
    unsigned char *const mine = sm + (a.bias ? (size_t)E * 4 : 0) + warp * lane_warp_bytes(E);
    float4 *const keys4 = reinterpret_cast<float4 *>(mine) + t * stride;
    LaneList &list = *reinterpret_cast<LaneList *>(mine + (size_t)8 * stride * 16);
    grid_dependency_wait();
    if (a.bias) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) reinterpret_cast<float *>(sm)[e] = clean_choice(__ldg(a.bias + e));
        __syncthreads();
    }
    const int ntok = a.g.R * a.g.T, ntask = (int)(((long long)ntok + 7) / 8);
    for (int task = blockIdx.x * nwarps + warp; task < ntask; task += gridDim.x * nwarps) {
        const long long u = (long long)task * 8 + t;
        const bool act = u < ntok && token_active(a.num_tokens, a.g.T, (int)u);
        if (!__any_sync(kAll, act)) continue;
        const float *const row = a.logits + (size_t)(act ? u : 0) * E;  // of a token that takes no part nothing is kept
        auto has = [&](int j) { return kFull || r + 4 * j < nu; };

        // 1. logits, then choices; NaN where there is none
        float4 v[NU];
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            if (!kFull) v[j] = make_float4(NAN, NAN, NAN, NAN);
            if (has(j)) {
                const uint4 b = ld_stream_v4(row + 4 * (r + 4 * j));
                v[j] = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
            }
        }
        const bool scored = a.bias && a.sigmoid;  // then an infinity needs no care
#pragma unroll
        for (int j = 0; j < NU; ++j)
            if (has(j))
#pragma unroll
                for (int c = 0; c < 4; ++c) part_of(v[j], c) = fmaxf(part_of(v[j], c), -FLT_MAX);
        if (!scored)
#pragma unroll
            for (int j = 0; j < NU; ++j)
                if (has(j))
#pragma unroll
                    for (int c = 0; c < 4; ++c) part_of(v[j], c) = fminf(part_of(v[j], c), FLT_MAX);
        float m = 0.0f, z = 1.0f, top = 1.0f;
        if (!a.sigmoid) {
            float4 x = make_float4(-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX);
#pragma unroll
            for (int j = 0; j < NU; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) part_of(x, c) = fmaxf(part_of(x, c), part_of(v[j], c));
            m = token_max(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
            if (a.bias || !a.renorm) {
                z = 0.0f;
#pragma unroll
                for (int j = 0; j < NU; ++j) {
                    float4 e = make_float4(fast_exp(v[j].x - m), fast_exp(v[j].y - m), fast_exp(v[j].z - m), fast_exp(v[j].w - m));
                    if (has(j)) z += (e.x + e.y) + (e.z + e.w);
                    if (a.bias) v[j] = e;
                }
                z = token_sum(z);
                top = __fdividef(1.0f, z);
            }
        }
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < NU; ++j)
                if (has(j)) {
                    float4 b = bias4[r + 4 * j];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        part_of(v[j], c) =
                            (a.sigmoid ? fast_sigmoid(part_of(v[j], c)) : part_of(v[j], c) * top) + part_of(b, c);
                }
        }
#pragma unroll
        for (int j = 0; j < NU; ++j)
            if (has(j)) keys4[r + 4 * j] = v[j];

        // 2. groups: which are kept, as bits, and which of this lane's units are theirs
        bool near = false;
        uint32_t units = ~0u;
        if constexpr (kGroups) {
            __syncwarp();
            const int upg = E / a.groups / 4, log_upg = 31 - __clz(upg);  // units per group: a power of two
            for (int g = r; g < a.groups; g += 4) {
                float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll 4
                for (int i = 0; i < upg; ++i) {
                    const float4 x = keys4[g * upg + ((i + r) & (upg - 1))];
                    const float h1 = fmaxf(x.x, x.y), l1 = fminf(x.x, x.y), h2 = fmaxf(x.z, x.w), l2 = fminf(x.z, x.w);
                    merge2(b1, b2, fmaxf(h1, h2), fmaxf(fminf(h1, h2), fmaxf(l1, l2)));
                }
                float value, off;
                group_value(a, b1, b2, m, top, value, off);
                list.key[t][g] = value;
                list.key[t][kLaneGroups + g] = off;
                const float q = a.best == 2 ? b2 : b1;  // below it by more than its error: none of the group's best
                list.best[t][g] = a.bias && !isinf(q) ? q - 4.0f * error_of(a.sigmoid, top, q) : q;
            }
            __syncwarp();
            uint32_t keep = 0;
            float lo = INFINITY, hi = -INFINITY;
            for (int g = r; g < a.groups; g += 4) {
                const float value = list.key[t][g], off = list.key[t][kLaneGroups + g];
                int before = 0;
#pragma unroll 4
                for (int q = 0; q < a.groups; ++q) {
                    const float other = list.key[t][q];
                    before += other > value || (other == value && q < g);
                }
                const bool in = before < a.kept;
                keep |= (uint32_t)in << g;
                if (in) lo = fminf(lo, value - off);
                else hi = fmaxf(hi, value + off);
            }
            __syncwarp();  // lanes of a token may have gone apart over their groups
            keep |= __shfl_xor_sync(kAll, keep, 1);
            keep |= __shfl_xor_sync(kAll, keep, 2);
            if (a.bias || a.best == 2) {
                const float least = -token_max(-lo), most = token_max(hi);  // by every lane
                near = act && !(least >= most);
                uint32_t open = __ballot_sync(kAll, near);
                if (open) {
                    while (open) {
                        const int s = (__ffs(open) - 1) >> 2;
                        open &= ~(15u << (4 * s));
                        const float *const token = reinterpret_cast<const float *>(mine) + (size_t)s * stride * 4;
                        const uint32_t exact = keep_exact(a, task * 8 + s, token, list.best[s], list.id[s], lane);
                        if (t == s) {
                            near = exact == ~0u;
                            keep = exact;
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < NU; ++j)  // so that they need not be held over the calls
                        if (has(j)) v[j] = keys4[r + 4 * j];
                }
            }
            units = 0;
#pragma unroll
            for (int j = 0; j < NU; ++j) units |= (keep >> ((r + 4 * j) >> log_upg) & 1) << j;
        }

        // 3. the bound
        float tau;
        {
            float c[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            // maxima of the kept units' components
#pragma unroll
            for (int j = 0; j < NU; ++j)
                if (!kGroups || (units >> j & 1))
#pragma unroll
                    for (int i = 0; i < 4; ++i) c[i] = fmaxf(c[i], part_of(v[j], i));
            if (L == 4) sort4(c);
            if (L == 2) {
                c[0] = fmaxf(c[0], c[2]);
                c[1] = fmaxf(c[1], c[3]);
                order2(c[0], c[1]);
            }
            if (L == 1) c[0] = fmaxf(fmaxf(c[0], c[1]), fmaxf(c[2], c[3]));
            float g[L];
#pragma unroll
            for (int i = 0; i < L; ++i) g[i] = c[i];
            tau = bound_of<KMAX>(g);
            if (a.bias && !isinf(tau)) tau -= 4.0f * error_of(a.sigmoid, top, tau);
        }

        // 4. candidates: as bits, then listed (a NaN is none)
        constexpr int kWords = (NU * 4 + 31) / 32;
        uint32_t bits[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w) bits[w] = 0;
#pragma unroll
        for (int j = 0; j < NU; ++j) {
            const float at = !kGroups || (units >> j & 1) ? tau : NAN;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (part_of(v[j], c) >= at) bits[j / 8] |= 1u << (j % 8 * 4 + c);
        }
        int cnt = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) cnt += __popc(bits[w]);
        const int side = __shfl_xor_sync(kAll, cnt, 1), two = cnt + side, rest = __shfl_xor_sync(kAll, two, 2);
        const int n = two + rest, listed = n < kList ? n : kList;
        int pos = (r & 1 ? side : 0) + (r & 2 ? rest : 0);
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            for (uint32_t b = bits[w]; b && pos < kList; b &= b - 1, ++pos) {
                const int i = w * 32 + __ffs(b) - 1, e = 4 * (r + 4 * (i >> 2)) + (i & 3);
                list.key[t][pos] = reinterpret_cast<const float *>(keys4)[e];
                list.id[t][pos] = e;
            }
        list.key[t][listed + r] = NAN;
#pragma unroll
        for (int i = 0; i < kRanks / 4; ++i) list.best[t][r + 4 * i] = NAN;
        __syncwarp();

        // 5. ranks
        constexpr int SL = (KMAX + 3) / 4;  // slots per lane
        int id[SL];
        // Places the candidates by rank and takes this lane's slots; false where that may not be the order.  by_id: of
        // equal choices the lower id first, right only for equal logits and biases, which are then compared.
        auto rank = [&](auto by_id) {
            constexpr bool kById = decltype(by_id)::value;
            for (int from = r; from < listed; from += 16) {
                float own[4];
                int above[4], own_id[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool there = from + 4 * i < listed;
                    own[i] = there ? list.key[t][from + 4 * i] : NAN;
                    if (kById) own_id[i] = there ? list.id[t][from + 4 * i] : 0;
                    above[i] = kById ? 0 : -1;  // each counts itself
                }
                for (int q = 0; q < listed; q += 4) {
                    float4 x = *reinterpret_cast<const float4 *>(&list.key[t][q]);
                    const uint32_t ids = kById ? *reinterpret_cast<const uint32_t *>(&list.id[t][q]) : 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float o = part_of(x, c);
                            if (kById) above[i] += o > own[i] || (o == own[i] && (int)(ids >> (8 * c) & 255) < own_id[i]);
                            else above[i] += o >= own[i];
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (from + 4 * i < listed && above[i] < (kById ? kRanks : k + 1)) {
                        list.best[t][above[i]] = own[i];
                        list.best_id[t][above[i]] = list.id[t][from + 4 * i];
                    }
            }
            __syncwarp();
            bool right = true;
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                const int j = r + 4 * i;
                id[i] = 0;
                if (j >= k) continue;
                const float c = list.best[t][j], next = list.best[t][j + 1];
                id[i] = list.best_id[t][j];
                bool good = c == c && !(a.bias && next != next && listed > j + 1);  // equal ones left the next rank empty
                if (a.bias && next == next && too_near(a.sigmoid, top, c, next)) {
                    good = false;
                    if (kById && act && c == next) {
                        const float *const bias = reinterpret_cast<const float *>(sm);
                        const float l0 = clean_logit(__ldg(row + id[i])), b0 = bias[id[i]];
                        auto alike = [&](int other) { return clean_logit(__ldg(row + other)) == l0 && bias[other] == b0; };
                        good = alike(list.best_id[t][j + 1]);
                        if (j == k - 1)  // the last slot answers for all behind it, and one alike says nothing of the next
                            for (int q = j + 2; good && q < listed; ++q) {
                                if (q < kRanks && !too_near(a.sigmoid, top, c, list.best[t][q])) break;
                                good = q < kRanks && alike(list.best_id[t][q]);
                            }
                    }
                }
                right = right && good;
            }
            return right;
        };
        bool again = !rank(std::false_type{});
        if (__any_sync(kAll, act && again && n <= kList)) again = !rank(std::true_type{});
        const bool whole = near || n > kList;
        const uint32_t again_all = __ballot_sync(kAll, act && (again || whole));
        const bool ok = act && !(again_all >> (lane & ~3) & 15);

        // gates
        float l[SL], e[SL];
#pragma unroll
        for (int i = 0; i < SL; ++i) l[i] = ok && r + 4 * i < k ? clean_logit(__ldg(row + id[i])) : 0.0f;
        if (a.renorm) {
            float high = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < SL; ++i)
                if (r + 4 * i < k) high = fmaxf(high, a.sigmoid ? fminf(l[i], 0.0f) : l[i]);
            high = token_max(high);
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                e[i] = r + 4 * i < k ? expf((a.sigmoid ? fminf(l[i], 0.0f) : l[i]) - high) : 0.0f;
                if (a.sigmoid) e[i] = __fdiv_rn(e[i], 1.0f + expf(-fabsf(l[i])));
                sum += e[i];
            }
            sum = token_sum(sum);
#pragma unroll
            for (int i = 0; i < SL; ++i) e[i] = a.scale * __fdiv_rn(e[i], sum);
        } else {
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                const float x = expf(a.sigmoid ? -fabsf(l[i]) : l[i] - m);
                e[i] = a.scale * (a.sigmoid ? __fdiv_rn(l[i] >= 0.0f ? 1.0f : x, 1.0f + x) : __fdiv_rn(x, z));
            }
        }
#pragma unroll
        for (int i = 0; i < SL; ++i)
            if (ok && r + 4 * i < k) {
                a.idx[(size_t)u * k + r + 4 * i] = id[i];
                a.gate[(size_t)u * k + r + 4 * i] = e[i];
            }
        // those the fp32 values left open: by their list, or from the start
        const uint32_t whole_all = __ballot_sync(kAll, act && whole);
        for (uint32_t left = again_all; left;) {
            const int s = (__ffs(left) - 1) >> 2;
            left &= ~(15u << (4 * s));
            if (!(whole_all >> (4 * s) & 15)) route_list(a, task * 8 + s, list, s, __shfl_sync(kAll, n, 4 * s), lane);
        }
        __syncwarp();
        for (uint32_t left = whole_all; left;) {  // these use the choices' room
            const int s = (__ffs(left) - 1) >> 2;
            left &= ~(15u << (4 * s));
            route_one(a, task * 8 + s, reinterpret_cast<long long *>(mine), lane);
        }
        __syncwarp();  // every lane is done with the warp's shared memory
    }
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

// The same for k up to 8 and E a multiple of 4: eight lanes per token, four tokens per warp, rows stored as 16-byte
// vectors.  65,536 x 256, top-8: 17.9 us (one warp per token 30) for 90 MB, of which 17 are 32-byte pieces around the chosen
// logits.  With the whole softmax (NU > 0) lane r holds units r, r + 8, ... of its token's row, E at most 32 * NU.
template <int NU>
__global__ void __launch_bounds__(32 * kWarps) route_scores_grad_lane_kernel(const ScoreArgs a) {
    extern __shared__ __align__(16) unsigned char sm[];
    const int E = a.g.E, k = a.g.k, nu = E / 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane >> 3, r = lane & 7;
    float *const row = reinterpret_cast<float *>(sm) + (size_t)(warp * 4 + t) * E;
    float4 *const row4 = reinterpret_cast<float4 *>(row);
    for (int c = r; c < nu; c += 8) row4[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
    grid_dependency_wait();
    auto sum8 = [](float v) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
        return v;
    };
    auto max8 = [](float v) {
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
        return v;
    };
    const int ntok = a.g.R * a.g.T, ntask = (int)(((long long)ntok + 3) / 4);
    // A task's ids and gradients are asked for two tasks ahead, their logits one task ahead.
    struct Slot {
        bool act;
        int id;
        float d;
    };
    auto ask = [&](int task) {
        const long long u = (long long)task * 4 + t;
        Slot s;
        s.act = task < ntask && u < ntok && token_active(a.num_tokens, a.g.T, (int)u);
        const bool slot = s.act && r < k;
        s.id = slot ? __ldg(a.idx + u * k + r) : -1;
        s.d = slot ? __ldg(a.d_gate + u * k + r) : 0.0f;
        return s;
    };
    auto logit = [&](int task, const Slot &s) {
        return (uint32_t)s.id < (uint32_t)E ? __ldg(a.logits + ((size_t)task * 4 + t) * E + s.id) : 0.0f;
    };
    const int step = gridDim.x * kWarps;
    int task = blockIdx.x * kWarps + warp;
    Slot now = ask(task), next = ask(task + step);
    float raw = logit(task, now);
    for (; task < ntask; task += step) {
        const bool act = now.act;
        const long long u = act ? (long long)task * 4 + t : 0;
        const float *const l = a.logits + (size_t)u * E;
        const int id = now.id;
        const bool in = (uint32_t)id < (uint32_t)E;
        if (act && r < k && !in) atomicOr(a.status, A2AV_DEV_BAD_EXPERT);
        const float d = in ? now.d : 0.0f, v = clean_logit(raw);
        now = next;
        raw = logit(task + step, now);
        next = ask(task + 2 * step);
        float4 x[NU > 0 ? NU : 1];
        if constexpr (NU > 0) {
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                x[j] = make_float4(-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX);
                if (act && r + 8 * j < nu) {
                    const uint4 b = ld_stream_v4(l + 4 * (r + 8 * j));
                    x[j] = make_float4(clean_logit(__uint_as_float(b.x)), clean_logit(__uint_as_float(b.y)),
                                       clean_logit(__uint_as_float(b.z)), clean_logit(__uint_as_float(b.w)));
                }
            }
        }
        const float ea = expf(-fabsf(v));
        const float rest = a.sigmoid ? __fdiv_rn(v >= 0.0f ? ea : 1.0f, 1.0f + ea) : 1.0f;  // 1 - s
        float val, sum = 0.0f, scale = 0.0f;
        if constexpr (NU > 0) {
            float m = -FLT_MAX, z = 0.0f;
#pragma unroll
            for (int j = 0; j < NU; ++j) m = fmaxf(m, fmaxf(fmaxf(x[j].x, x[j].y), fmaxf(x[j].z, x[j].w)));
            m = max8(m);
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                x[j] = make_float4(expf(x[j].x - m), expf(x[j].y - m), expf(x[j].z - m), expf(x[j].w - m));
                if (r + 8 * j < nu) z += (x[j].x + x[j].y) + (x[j].z + x[j].w);
            }
            z = sum8(z);
            val = in ? a.scale * d * __fdiv_rn(expf(v - m), z) : 0.0f;
            sum = sum8(val);
            scale = __fdiv_rn(1.0f, z);
        } else if (a.renorm) {
            const float base = a.sigmoid ? fminf(v, 0.0f) : v, high = max8(in ? base : -INFINITY);
            float e = in ? expf(base - high) : 0.0f;
            if (a.sigmoid) e = __fdiv_rn(e, 1.0f + ea);
            const float all = sum8(e), g = in ? __fdiv_rn(e, all) : 0.0f, dot = sum8(g * d);
            val = in ? a.scale * g * (d - dot) * rest : 0.0f;
        } else {
            val = in ? a.scale * d * __fdiv_rn(v >= 0.0f ? 1.0f : ea, 1.0f + ea) * rest : 0.0f;
        }
        // an id that occurs twice: all its slots' values, added in slot order by each of them
        bool twice = false;
#pragma unroll
        for (int o = 1; o < 8; ++o) twice |= __shfl_xor_sync(kAll, id, o) == id;
        if (__any_sync(kAll, in && twice)) {
            float all = 0.0f;
            for (int j = 0; j < 8; ++j) {
                const int other = __shfl_sync(kAll, id, (lane & ~7) + j);
                const float w = __shfl_sync(kAll, val, (lane & ~7) + j);
                if (other == id) all += w;
            }
            val = all;
        }
        if (in) row[id] = val;
        __syncwarp();
        float4 *const out = reinterpret_cast<float4 *>(a.d_logits + (size_t)u * E);
        if constexpr (NU > 0) {
#pragma unroll
            for (int j = 0; j < NU; ++j)
                if (act && r + 8 * j < nu) {
                    const float4 w = row4[r + 8 * j];
                    out[r + 8 * j] = make_float4(w.x - sum * (x[j].x * scale), w.y - sum * (x[j].y * scale),
                                                 w.z - sum * (x[j].z * scale), w.w - sum * (x[j].w * scale));
                }
        } else if (act) {
#pragma unroll 4
            for (int c = r; c < nu; c += 8) out[c] = row4[c];
        }
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

template <int NU>
cudaError_t launch_grad_lanes(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = route_scores_grad_lane_kernel<NU>;
    const cudaError_t e = allow_smem(kernel, done, p.cfg.device, (size_t)kWarps * 16 * kMaxExperts);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)kWarps * 16 * a.g.E;
    const int ntask = (int)(((long long)a.g.R * a.g.T + 3) / 4), want = (ntask + kWarps - 1) / kWarps;
    const int fit = (int)(220 * 1024 / (smem + 1024)), cap = p.num_sms * (fit < 12 ? fit : 12);
    return launch_pdl(kernel, want < cap ? want : cap, 32 * kWarps, smem, s, a);
}

template <int NU, int KMAX, bool kGroups, bool kFull>
cudaError_t launch_lanes(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = route_scores_lane_kernel<NU, KMAX, kGroups, kFull>;
    const auto bytes = [](int E, int warps) { return (size_t)E * 4 + warps * lane_warp_bytes(E); };
    const cudaError_t e = allow_smem(kernel, done, p.cfg.device, bytes(16 * NU, kWarps));
    if (e != cudaSuccess) return e;
    // few tokens: a warp per block, so that they spread over the SMs
    const int ntask = (int)(((long long)a.g.R * a.g.T + 7) / 8), warps = ntask <= kWarps * p.num_sms ? 1 : kWarps;
    const int want = (ntask + warps - 1) / warps, cap = p.num_sms * (4 * kWarps / warps);
    return launch_pdl(kernel, want < cap ? want : cap, 32 * warps, bytes(a.g.E, warps), s, a);
}

template <int NU, bool kFull>
cudaError_t launch_lanes_k(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s) {
    if (a.g.k <= 1) return launch_lanes<NU, 1, false, kFull>(p, a, s);
    if (a.g.k <= 2) return launch_lanes<NU, 2, false, kFull>(p, a, s);
    if (a.g.k <= 4) return launch_lanes<NU, 4, false, kFull>(p, a, s);
    return launch_lanes<NU, 8, false, kFull>(p, a, s);
}

}  // namespace

cudaError_t launch_route_scores(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s) {
    const int E = a.g.E, G = a.kept < a.groups ? a.groups : 1;
    if (a.g.k <= 8 && E <= 256 && E % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0) {
        if (G == 1) {
            if (E <= 16) return launch_lanes_k<1, false>(p, a, s);
            if (E <= 32) return launch_lanes_k<2, false>(p, a, s);
            if (E <= 64) return launch_lanes_k<4, false>(p, a, s);
            if (E < 128) return launch_lanes_k<8, false>(p, a, s);
            if (E == 128) return launch_lanes_k<8, true>(p, a, s);
            if (E < 256) return launch_lanes_k<16, false>(p, a, s);
            return launch_lanes_k<16, true>(p, a, s);
        }
        // groups of whole units, their number a power of two
        const int upg = E / G / 4;
        if (G <= kLaneGroups && E % (4 * G) == 0 && (upg & (upg - 1)) == 0) {
            if (E <= 64) return launch_lanes<4, 8, true, false>(p, a, s);
            if (E <= 128) return launch_lanes<8, 8, true, false>(p, a, s);
            return E == 256 ? launch_lanes<16, 8, true, true>(p, a, s) : launch_lanes<16, 8, true, false>(p, a, s);
        }
    }
    static std::atomic<uint64_t> done{0};
    return launch_tokens(route_scores_kernel, done, sizeof(long long), p, a, s);
}

cudaError_t launch_route_scores_grad(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s) {
    const int E = a.g.E;
    if (a.g.k <= 8 && E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.d_logits)) % 16 == 0) {
        if (a.sigmoid || a.renorm) return launch_grad_lanes<0>(p, a, s);
        if (E <= 32) return launch_grad_lanes<1>(p, a, s);
        if (E <= 64) return launch_grad_lanes<2>(p, a, s);
        if (E <= 128) return launch_grad_lanes<4>(p, a, s);
        if (E <= 256) return launch_grad_lanes<8>(p, a, s);
    }
    static std::atomic<uint64_t> done{0};
    return launch_tokens(route_scores_grad_kernel, done, sizeof(float), p, a, s);
}

}  // namespace a2av
