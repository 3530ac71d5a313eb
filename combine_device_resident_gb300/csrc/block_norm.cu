// The norms before and after a block with its gate and the residual's scale,
// and their gradient.
//
//   u = x * r1 * post,            r1 = 1 / sqrt(mean x^2 + eps)
//   z = a * residual + b * gate * u,   residual_out = bf16(z)
//   v = z * weight * r2,          r2 = 1 / sqrt(mean z^2 + eps)
//
// One block per row at a time, the row in registers between its uses, so every
// tensor is read once.  Bound by HBM.
//
// Gradient, dy and dr those of v and of residual_out, n = x * r1:
//   dv = dy * weight;  dz = dr + r2 * dv - z * (r2^3 * mean(dv z));  d_residual = a * dz
//   db = b * dz;  d_gate = db * u;  du = db * gate
//   dn = du * post;  dx = r1 * dn - x * (r1^3 * mean(dn x))
//   d_weight = sum dy * z * r2,  d_post = sum du * n   over the tokens
// z and the roots are taken again from x and residual: three block sums, each
// after the one before.  A block takes consecutive rows; its threads keep their
// columns, so the sums over the tokens are each thread's own in shared memory;
// the blocks' sums are added by a second kernel in a fixed order.
#include "block_ops.cuh"
#include "expert_common.cuh"
#include "row_math.cuh"

namespace a2av {
namespace {

constexpr int kMaxWarps = 32;

__device__ __forceinline__ bool row_active(const BlockNormArgs &a, long long row) {
    if (!a.num_tokens) return true;
    const int s = (int)(row / a.g.T);
    return row - (long long)s * a.g.T < active_tokens(a.num_tokens, s, a.g.T);
}

// The gate's row of a token.
__device__ __forceinline__ const uint16_t *gate_row(const BlockNormArgs &a, long long row) {
    const size_t H = a.g.H;
    return a.gate + (a.gate_kind == A2AV_GATE_TOKEN  ? (size_t)row * H
                     : a.gate_kind == A2AV_GATE_RANK ? (size_t)(row / a.g.T) * H
                                                     : 0);
}

// Two fp32 values in a register pair, for the two-lane instructions.
using pair = uint64_t;
__device__ __forceinline__ pair both(float lo, float hi) {
    pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ pair both(float v) { return both(v, v); }
__device__ __forceinline__ void split(pair p, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ pair mul2(pair a, pair b) {
    pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair add2(pair a, pair b) {
    pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ pair fma2(pair a, pair b, pair c) {
    pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float sum2(pair p) {
    float lo, hi;
    split(p, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ uint32_t bf16_of(pair p) {
    float lo, hi;
    split(p, lo, hi);
    return bf16x2(lo, hi);
}
// Eight bf16 values as four pairs, and back.
__device__ __forceinline__ void unpack8(const uint4 &v, pair (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = both(lo_f(w[i]), hi_f(w[i]));
}
__device__ __forceinline__ uint4 pack8(const pair (&f)[4]) {
    return make_uint4(bf16_of(f[0]), bf16_of(f[1]), bf16_of(f[2]), bf16_of(f[3]));
}

// A row of fp32 in shared memory, eight values of a vector apart in two halves, so that a warp's 16-byte accesses lie
// on consecutive 16 bytes.  A thread touches its own columns alone.
__device__ __forceinline__ void ld_shared(const ulonglong2 *row, int nvec, int i, pair (&f)[4]) {
    const ulonglong2 lo = row[i], hi = row[nvec + i];
    f[0] = lo.x, f[1] = lo.y, f[2] = hi.x, f[3] = hi.y;
}
__device__ __forceinline__ void st_shared(ulonglong2 *row, int nvec, int i, const pair (&f)[4]) {
    row[i] = make_ulonglong2(f[0], f[1]);
    row[nvec + i] = make_ulonglong2(f[2], f[3]);
}

// Brings `bytes` (a multiple of 16) into L2.
__device__ __forceinline__ void prefetch_row(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Over the block: sum of s, and of t its sum or maximum (NaN kept).  `part` is free again after the next barrier.
template <bool kMax>
__device__ __forceinline__ void block_reduce(float &s, float &t, float (*part)[kMaxWarps]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    s = warp_sum(s);
    t = kMax ? warp_max_nan(t) : warp_sum(t);
    if (lane == 0) {
        part[0][warp] = s;
        part[1][warp] = t;
    }
    __syncthreads();
    s = warp_sum(lane < nwarps ? part[0][lane] : 0.0f);
    t = lane < nwarps ? part[1][lane] : 0.0f;
    t = kMax ? warp_max_nan(t) : warp_sum(t);
}

// A weight: the same for every row, so it stays in the L1 cache.
__device__ __forceinline__ uint4 ld_weight(const uint16_t *w, int i) {
    return __ldg(reinterpret_cast<const uint4 *>(w) + i);
}

// The factor of x * r1 in z, per channel: branch_scale * post * gate, the gate left out where it is the token's own
// (gate null here).
__device__ __forceinline__ void set_coef(const BlockNormArgs &a, const uint16_t *gate, ulonglong2 *coef) {
    const int nvec = a.g.H / 8;
    for (int i = threadIdx.x; i < nvec; i += blockDim.x) {
        pair c[4], w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = both(a.branch_scale);
        if (a.post) {
            unpack8(ld_weight(a.post, i), w);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = mul2(c[e], w[e]);
        }
        if (gate) {
            unpack8(ld_weight(gate, i), w);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = mul2(c[e], w[e]);
        }
        st_shared(coef, nvec, i, c);
    }
}

constexpr int kV = 2;  // 16-byte vectors of a row per thread

// The next row's loads are in registers while a row is worked on.  kBlocks blocks fit an SM.
template <int V, int kThreads, int kBlocks, bool kPost, bool kToken>
__global__ void __launch_bounds__(kThreads, kBlocks) block_norm_kernel(const BlockNormArgs a) {
    extern __shared__ __align__(16) ulonglong2 coef[];  // [half of a vector][vector]
    __shared__ float part[2][2][2][kMaxWarps];          // [which sum][row parity]
    const int H = a.g.H, nvec = H / 8, tid = threadIdx.x, width = blockDim.x;
    const long long rows = (long long)a.g.R * a.g.T;
    const float inv_h = 1.0f / (float)H;
    const pair alpha = both(a.residual_scale);
    grid_dependency_wait();
    int parity = 0;
    uint4 xv[V], rv[V], gv[V];
    long long row = blockIdx.x;
    auto load = [&] {  // from the first row on that takes part
        while (row < rows && !row_active(a, row)) row += gridDim.x;
        if (row >= rows) return;
        const size_t at = (size_t)row * H;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            xv[j] = i < nvec ? ld_row(a.x + at + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
            rv[j] = i < nvec ? ld_row(a.residual + at + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
            if (kToken) gv[j] = i < nvec ? ld_row(a.gate + at + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
        }
    };
    load();
    const uint16_t *coef_of = nullptr;
    if (row < rows) set_coef(a, coef_of = kToken || !a.gate ? nullptr : gate_row(a, row), coef);
    while (row < rows) {
        const size_t at = (size_t)row * H;
        if (!kToken && a.gate_kind == A2AV_GATE_RANK && gate_row(a, row) != coef_of)
            set_coef(a, coef_of = gate_row(a, row), coef);
        uint8_t *q = a.rows8 ? a.rows8 + (size_t)row * (H + 16) : nullptr;
        pair z[V][4];
        float sum = 0.0f, peak = 0.0f, r1 = 1.0f;
        if (kPost) {
            pair s = both(0.0f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                pair x[4];
                unpack8(xv[j], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fma2(x[e], x[e], s);
            }
            sum = sum2(s);
            block_reduce<false>(sum, peak, part[0][parity]);
            r1 = 1.0f / sqrtf(sum * inv_h + a.eps);
        }
        peak = 0.0f;
        pair s = both(0.0f);
        const pair root = both(r1);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) continue;
            pair x[4], c[4];
            unpack8(xv[j], x);
            unpack8(rv[j], z[j]);
            ld_shared(coef, nvec, i, c);
            if (kToken) {
                pair g[4];
                unpack8(gv[j], g);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = mul2(c[e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[j][e] = fma2(kPost ? mul2(x[e], root) : x[e], c[e], mul2(z[j][e], alpha));
                s = fma2(z[j][e], z[j][e], s);
            }
            if (a.residual_out) st_v4(a.residual_out + at + (size_t)i * 8, pack8(z[j]));
            if (a.weight) {
                pair w[4];
                unpack8(ld_weight(a.weight, i), w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[j][e] = mul2(z[j][e], w[e]);
                    if (a.rows8) {
                        float lo, hi;
                        split(z[j][e], lo, hi);
                        peak = max_nan(peak, max_nan(fabsf(lo), fabsf(hi)));
                    }
                }
            }
        }
        row += gridDim.x;
        load();
        if (a.weight) {
            sum = sum2(s);
            block_reduce<true>(sum, peak, part[1][parity]);
            const float r2 = 1.0f / sqrtf(sum * inv_h + a.eps);
            peak *= r2;
            const bool zero = peak < kZeroRow;  // false for NaN
            const float inv = zero ? 0.0f : kLow8 / peak;
            if (q && tid == 0) st_v4(q + H, make_uint4(__float_as_uint(zero ? 0.0f : peak / kLow8), 0, 0, 0));
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int i = tid + j * width;
                if (i >= nvec) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) z[j][e] = mul2(z[j][e], both(r2));
                if (a.y) st_v4(a.y + at + (size_t)i * 8, pack8(z[j]));
                if (q) {
                    uint32_t b[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float lo, hi;
                        split(mul2(z[j][e], both(inv)), lo, hi);
                        b[e] = e4m3x2(lo, hi);
                    }
                    *reinterpret_cast<uint2 *>(q + (size_t)i * 8) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
                }
            }
        }
        parity ^= 1;
    }
}

// ---- the gradient ----------------------------------------------------------------

// The sums over the tokens a block keeps: dy * z * r2, and dz * n, out of which both d_post (times b and the gate) and
// d_gate (times b and post) come, as the gate is the same for all of the block's rows; with a gate per token dz * gate * n.
enum { kSumWeight, kSumBranch, kSums };

// Rows of block b: consecutive, and of one rank where the gate is per rank and its products are summed.
__device__ __host__ inline void block_rows(const Geometry &g, bool per_rank, int blocks, int b, long long &first,
                                           long long &end) {
    const int parts = per_rank ? blocks / g.R : blocks;
    const long long rows = per_rank ? g.T : (long long)g.R * g.T;
    const int rank = per_rank ? b / parts : 0, c = b - rank * parts;
    first = rank * rows + rows * c / parts;
    end = rank * rows + rows * (c + 1) / parts;
}

__device__ __forceinline__ bool sum_branch(const BlockNormArgs &a) {
    return a.d_post || (a.d_gate && a.gate_kind != A2AV_GATE_TOKEN);
}

template <int V, int kThreads, int kBlocks, bool kPost, bool kToken>
__global__ void __launch_bounds__(kThreads, kBlocks) block_norm_grad_kernel(const BlockNormArgs a, bool per_rank) {
    extern __shared__ __align__(16) ulonglong2 coef[];  // then the sums, each [half of a vector][vector]
    __shared__ float part[3][2][2][kMaxWarps];
    const int H = a.g.H, nvec = H / 8, tid = threadIdx.x, width = blockDim.x;
    const bool branch = sum_branch(a);
    ulonglong2 *const acc = coef + 2 * nvec;
    {
        const pair zero[4] = {0, 0, 0, 0};
        for (int i = tid; i < nvec; i += width)
            for (int q = 0; q < kSums; ++q) st_shared(acc + q * 2 * nvec, nvec, i, zero);
    }
    long long row, end;
    block_rows(a.g, per_rank, gridDim.x, blockIdx.x, row, end);
    grid_dependency_wait();
    int parity = 0;
    const float inv_h = 1.0f / (float)H;
    const pair alpha = both(a.residual_scale);
    const uint16_t *coef_of = nullptr;
    bool coef_set = false;
    for (; row < end; ++row) {
        if (!row_active(a, row)) continue;
        const size_t at = (size_t)row * H;
        const uint16_t *gate = kToken || !a.gate ? nullptr : gate_row(a, row);
        if (!coef_set || gate != coef_of) {
            set_coef(a, coef_of = gate, coef);
            coef_set = true;
        }
        const uint4 none = make_uint4(0, 0, 0, 0);
        uint4 xv[V], rv[V], dyv[V], drv[V], gv[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            const bool in = i < nvec;
            xv[j] = in ? ld_row(a.x + at + (size_t)i * 8) : none;
            rv[j] = in ? ld_row(a.residual + at + (size_t)i * 8) : none;
            dyv[j] = in && a.d_y ? ld_row(a.d_y + at + (size_t)i * 8) : none;
            drv[j] = in && a.d_residual_out ? ld_row(a.d_residual_out + at + (size_t)i * 8) : none;
            if (kToken) gv[j] = in ? ld_row(a.gate + at + (size_t)i * 8) : none;
        }
        if (row + 1 < end && tid < 5) {  // the next row on its way into L2
            const uint16_t *from = tid == 0   ? a.x
                                   : tid == 1 ? a.residual
                                   : tid == 2 ? a.d_y
                                   : tid == 3 ? a.d_residual_out
                                   : kToken   ? a.gate
                                              : nullptr;
            if (from) prefetch_row(from + at + H, 2 * H);
        }
        float r1 = 1.0f, unused = 0.0f;
        if (kPost) {
            pair s = both(0.0f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                pair x[4];
                unpack8(xv[j], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fma2(x[e], x[e], s);
            }
            float sum = sum2(s);
            block_reduce<false>(sum, unused, part[0][parity]);
            r1 = 1.0f / sqrtf(sum * inv_h + a.eps);
        }
        pair z[V][4], zz2 = both(0.0f), vz2 = both(0.0f);
        const pair root1 = both(r1);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) continue;
            pair x[4], c[4];
            unpack8(xv[j], x);
            unpack8(rv[j], z[j]);
            ld_shared(coef, nvec, i, c);
            if (kToken) {
                pair g[4];
                unpack8(gv[j], g);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = mul2(c[e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[j][e] = fma2(kPost ? mul2(x[e], root1) : x[e], c[e], mul2(z[j][e], alpha));
                zz2 = fma2(z[j][e], z[j][e], zz2);
            }
            if (a.d_y) {
                pair w[4], dy[4];
                unpack8(ld_weight(a.weight, i), w);
                unpack8(dyv[j], dy);
#pragma unroll
                for (int e = 0; e < 4; ++e) vz2 = fma2(mul2(dy[e], w[e]), z[j][e], vz2);
            }
        }
        float r2 = 0.0f, c2 = 0.0f;
        if (a.d_y) {
            float zz = sum2(zz2), vz = sum2(vz2);
            block_reduce<false>(zz, vz, part[1][parity]);
            r2 = 1.0f / sqrtf(zz * inv_h + a.eps);
            c2 = r2 * r2 * r2 * (vz * inv_h);
        }
        const pair root2 = both(r2), less2 = both(-c2);
        pair nx2 = both(0.0f);
        pair(&dn)[V][4] = z;  // z's place takes dz * coef: the gradient of n = x * r1
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) continue;
            pair dz[4], x[4], c[4];
            unpack8(drv[j], dz);
            if (a.d_y) {
                pair dy[4], w[4];
                unpack8(dyv[j], dy);
                if (a.d_weight) {
                    pair t[4];
                    ld_shared(acc + kSumWeight * 2 * nvec, nvec, i, t);
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[e] = fma2(dy[e], mul2(z[j][e], root2), t[e]);
                    st_shared(acc + kSumWeight * 2 * nvec, nvec, i, t);
                }
                unpack8(ld_weight(a.weight, i), w);
#pragma unroll
                for (int e = 0; e < 4; ++e) dz[e] = fma2(less2, z[j][e], fma2(mul2(dy[e], w[e]), root2, dz[e]));
            }
            {
                pair t[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = mul2(dz[e], alpha);
                st_v4(a.d_residual + at + (size_t)i * 8, pack8(t));
            }
            unpack8(xv[j], x);
            if (branch) {
                pair t[4], g[4];
                ld_shared(acc + kSumBranch * 2 * nvec, nvec, i, t);
                if (kToken) unpack8(gv[j], g);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    t[e] = fma2(kToken ? mul2(dz[e], g[e]) : dz[e], kPost ? mul2(x[e], root1) : x[e], t[e]);
                st_shared(acc + kSumBranch * 2 * nvec, nvec, i, t);
            }
            ld_shared(coef, nvec, i, c);
            if (kToken) {
                if (a.d_gate) {  // b * dz * u
                    pair t[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[e] = mul2(mul2(dz[e], c[e]), kPost ? mul2(x[e], root1) : x[e]);
                    st_v4(static_cast<uint16_t *>(a.d_gate) + at + (size_t)i * 8, pack8(t));
                }
                pair g[4];
                unpack8(gv[j], g);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = mul2(c[e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dn[j][e] = mul2(dz[e], c[e]);
                if (kPost) nx2 = fma2(dn[j][e], x[e], nx2);
            }
        }
        float c1 = 0.0f;
        if (kPost) {
            float nx = sum2(nx2);
            block_reduce<false>(nx, unused, part[2][parity]);
            c1 = r1 * r1 * r1 * (nx * inv_h);
        }
        const pair less1 = both(-c1);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) continue;
            pair x[4];
            unpack8(xv[j], x);
            if (kPost) {
#pragma unroll
                for (int e = 0; e < 4; ++e) dn[j][e] = fma2(dn[j][e], root1, mul2(x[e], less1));
            }
            st_v4(a.d_x + at + (size_t)i * 8, pack8(dn[j]));
        }
        parity ^= 1;
    }
    for (int q = 0; q < kSums; ++q)
        if (q == kSumWeight ? a.d_weight != nullptr : branch)
            for (int i = tid; i < nvec; i += width) {
                ulonglong2 *out = reinterpret_cast<ulonglong2 *>(a.scratch + ((size_t)blockIdx.x * kSums + q) * H) + 2 * i;
                out[0] = acc[(q * 2) * nvec + i];
                out[1] = acc[(q * 2 + 1) * nvec + i];
            }
}

// The blocks' sums S added up: d_weight = sum S, d_post = b * sum gate * S, d_gate = b * post * sum S (per rank over its
// blocks).
// The blocks in eight shares, each in order, then the shares in order.
enum { kOutWeight, kOutPost, kOutGate };
constexpr int kSumWarps = 8;

__global__ void __launch_bounds__(32 * kSumWarps) norm_sums_kernel(const BlockNormArgs a, int blocks, bool per_rank) {
    __shared__ float4 part[kSumWarps][32];
    const int H = a.g.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;  // four columns
    const int q = blockIdx.y < kOutGate ? blockIdx.y : kOutGate, rank = blockIdx.y - q;
    float *out = q == kOutWeight ? a.d_weight : q == kOutPost ? a.d_post : static_cast<float *>(a.d_gate);
    grid_dependency_wait();
    if (!out) return;
    const bool shared_gate = a.gate && (a.gate_kind == A2AV_GATE_CHANNEL || per_rank);
    const int parts = per_rank ? blocks / a.g.R : blocks;  // of one gate
    const int n = q == kOutGate ? parts : blocks, b0 = rank * parts;
    auto weight4 = [&](const uint16_t *w, size_t row) {
        const uint2 v = *(reinterpret_cast<const uint2 *>(w + row * H) + i);
        return make_float4(lo_f(v.x), hi_f(v.x), lo_f(v.y), hi_f(v.y));
    };
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < H / 4) {
        const float *from = a.scratch + (size_t)(q == kOutWeight ? kSumWeight : kSumBranch) * H;
#pragma unroll 8
        for (int b = (int)((long long)n * warp / kSumWarps); b < (int)((long long)n * (warp + 1) / kSumWarps); ++b) {
            float4 v = *(reinterpret_cast<const float4 *>(from + (size_t)(b0 + b) * kSums * H) + i);
            if (q == kOutPost && per_rank) {
                const float4 w = weight4(a.gate, b / parts);
                v.x *= w.x, v.y *= w.y, v.z *= w.z, v.w *= w.w;
            }
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < H / 4) {
        for (int w = 1; w < kSumWarps; ++w) {
            const float4 v = part[w][lane];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const uint16_t *times = q == kOutGate ? a.post : q == kOutPost && shared_gate && !per_rank ? a.gate : nullptr;
        if (times) {
            const float4 w = weight4(times, 0);
            s.x *= w.x, s.y *= w.y, s.z *= w.z, s.w *= w.w;
        }
        const float b = q == kOutWeight ? 1.0f : a.branch_scale;
        s.x *= b, s.y *= b, s.z *= b, s.w *= b;
        reinterpret_cast<float4 *>(out + (size_t)rank * H)[i] = s;
    }
}

int row_threads(int H, int V) { return ((H / 8 + V - 1) / V + 31) / 32 * 32; }

// Whether the gradient's blocks keep to a rank each.
bool keeps_to_rank(const BlockNormArgs &a) {
    return a.gate_kind == A2AV_GATE_RANK && (a.d_gate || a.d_post);
}

// Blocks of `threads` threads and `smem` bytes each that an SM holds, the kernels' registers allowing 1,024 threads.
int blocks_per_sm(int threads, size_t smem) {
    const int by_threads = threads > 512 ? 1 : 1024 / threads, by_smem = (int)(228 * 1024 / (smem + 3 * 1024));
    const int n = by_threads < by_smem ? by_threads : by_smem;
    return n < 1 ? 1 : n > 16 ? 16 : n;
}
size_t coef_bytes(int H) { return (size_t)H * sizeof(float); }
size_t grad_smem(int H) { return coef_bytes(H) * (1 + kSums); }

// Blocks of the gradient: what the SMs hold, at most one per row, a multiple of R where each is to keep to a rank.
int grad_blocks(int num_sms, const Geometry &g, bool per_rank) {
    const long long rows = (long long)g.R * g.T;
    const long long most = (long long)num_sms * blocks_per_sm(row_threads(g.H, kV), grad_smem(g.H));
    if (!per_rank) return (int)(rows < most ? rows : most);
    const long long parts = most / g.R < 1 ? 1 : most / g.R;
    return g.R * (int)(g.T < parts ? g.T : parts);
}

template <int V, int kThreads, int kBlocks, bool kPost, bool kToken>
cudaError_t launch_norm(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = block_norm_kernel<V, kThreads, kBlocks, kPost, kToken>;
    const size_t smem = coef_bytes(a.g.H);
    const cudaError_t e = allow_smem(kernel, done, p.cfg.device, coef_bytes(kMaxNormRow));
    if (e != cudaSuccess) return e;
    const int threads = row_threads(a.g.H, V);
    const long long rows = (long long)a.g.R * a.g.T, cap = (long long)p.num_sms * blocks_per_sm(threads, smem);
    return launch_pdl(kernel, (int)(rows < cap ? rows : cap), threads, smem, s, a);
}

template <bool kPost, bool kToken>
cudaError_t launch_norm_rows(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    if (a.g.H > 16384) return launch_norm<4, 1024, 1, kPost, kToken>(p, a, s);
    if (a.g.H > 8192) return launch_norm<kV, 1024, 1, kPost, kToken>(p, a, s);
    return launch_norm<kV, 512, 2, kPost, kToken>(p, a, s);
}

template <int V, int kThreads, int kBlocks, bool kPost, bool kToken>
cudaError_t launch_grad(const a2av_plan_s &p, const BlockNormArgs &a, int blocks, bool per_rank, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = block_norm_grad_kernel<V, kThreads, kBlocks, kPost, kToken>;
    const cudaError_t e = allow_smem(kernel, done, p.cfg.device, grad_smem(kMaxNormGradRow));
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, blocks, row_threads(a.g.H, V), grad_smem(a.g.H), s, a, per_rank);
}

template <bool kPost, bool kToken>
cudaError_t launch_grad_rows(const a2av_plan_s &p, const BlockNormArgs &a, int blocks, bool per_rank, cudaStream_t s) {
    if (a.g.H > 8192) return launch_grad<kV, 1024, 1, kPost, kToken>(p, a, blocks, per_rank, s);
    if (a.g.H > 7168) return launch_grad<kV, 512, 2, kPost, kToken>(p, a, blocks, per_rank, s);
    return launch_grad<kV, 448, 2, kPost, kToken>(p, a, blocks, per_rank, s);  // room for 72 registers
}

}  // namespace

cudaError_t launch_block_norm(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    const bool token = a.gate_kind == A2AV_GATE_TOKEN;
    if (a.post) return token ? launch_norm_rows<true, true>(p, a, s) : launch_norm_rows<true, false>(p, a, s);
    return token ? launch_norm_rows<false, true>(p, a, s) : launch_norm_rows<false, false>(p, a, s);
}

int64_t norm_scratch_bytes(const a2av_plan_s &p) {
    const int one = grad_blocks(p.num_sms, p.g, false), ranks = grad_blocks(p.num_sms, p.g, true);
    return (int64_t)(one > ranks ? one : ranks) * kSums * p.g.H * (int64_t)sizeof(float);
}

cudaError_t launch_block_norm_grad(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s, int64_t &launches) {
    const bool per_rank = keeps_to_rank(a);
    const bool sums = a.d_weight || a.d_post || (a.d_gate && a.gate_kind != A2AV_GATE_TOKEN);
    const int blocks = grad_blocks(p.num_sms, a.g, per_rank);
    const bool token = a.gate_kind == A2AV_GATE_TOKEN;
    cudaError_t e = a.post ? (token ? launch_grad_rows<true, true>(p, a, blocks, per_rank, s)
                                    : launch_grad_rows<true, false>(p, a, blocks, per_rank, s))
                           : (token ? launch_grad_rows<false, true>(p, a, blocks, per_rank, s)
                                    : launch_grad_rows<false, false>(p, a, blocks, per_rank, s));
    if (e != cudaSuccess) return e;
    ++launches;
    if (!sums) return cudaSuccess;
    BlockNormArgs b = a;
    if (token) b.d_gate = nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.g.H / 4 + 31) / 32, kOutGate + (per_rank ? a.g.R : 1));
    cfg.blockDim = dim3(32 * kSumWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, norm_sums_kernel, b, blocks, per_rank);
    if (e == cudaSuccess) ++launches;
    return e;
}

}  // namespace a2av
