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

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = lo_f(w[i]);
        f[2 * i + 1] = hi_f(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
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

constexpr int kV = 2;  // 16-byte vectors of a row per thread

// The next row's loads are in registers while a row is worked on.  kBlocks blocks fit an SM.
template <int V, int kThreads, int kBlocks, bool kPost>
__global__ void __launch_bounds__(kThreads, kBlocks) block_norm_kernel(const BlockNormArgs a) {
    __shared__ float part[2][2][2][kMaxWarps];  // [which sum][row parity]
    const int H = a.g.H, nvec = H / 8, tid = threadIdx.x, width = blockDim.x;
    const long long rows = (long long)a.g.R * a.g.T;
    const float inv_h = 1.0f / (float)H;
    grid_dependency_wait();
    int parity = 0;
    uint4 xv[V], rv[V];
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
        }
    };
    load();
    while (row < rows) {
        const size_t at = (size_t)row * H;
        const uint16_t *gate = a.gate ? gate_row(a, row) : nullptr;
        uint8_t *q = a.rows8 ? a.rows8 + (size_t)row * (H + 16) : nullptr;
        float z[V][8];
        float sum = 0.0f, peak = 0.0f, r1 = 1.0f;
        if (kPost) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float x[8];
                unpack8(xv[j], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
            }
            block_reduce<false>(sum, peak, part[0][parity]);
            r1 = 1.0f / sqrtf(sum * inv_h + a.eps);
        }
        sum = 0.0f;
        peak = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            float x[8], w[8];
            unpack8(xv[j], x);
            unpack8(rv[j], z[j]);
            if (i >= nvec) continue;
            if (kPost) {
                unpack8(ld_weight(a.post, i), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * r1 * w[e];
            }
            if (gate) {
                unpack8(ld_weight(gate, i), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[j][e] = fmaf(a.branch_scale, x[e], a.residual_scale * z[j][e]);
                sum = fmaf(z[j][e], z[j][e], sum);
            }
            if (a.residual_out) st_v4(a.residual_out + at + (size_t)i * 8, pack8(z[j]));
            if (a.weight) {
                unpack8(ld_weight(a.weight, i), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    z[j][e] *= w[e];
                    if (a.rows8) peak = max_nan(peak, fabsf(z[j][e]));
                }
            }
        }
        row += gridDim.x;
        load();
        if (a.weight) {
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
                for (int e = 0; e < 8; ++e) z[j][e] *= r2;
                if (a.y) st_v4(a.y + at + (size_t)i * 8, pack8(z[j]));
                if (q) {
                    uint2 v;
                    v.x = e4m3x2(z[j][0] * inv, z[j][1] * inv) | e4m3x2(z[j][2] * inv, z[j][3] * inv) << 16;
                    v.y = e4m3x2(z[j][4] * inv, z[j][5] * inv) | e4m3x2(z[j][6] * inv, z[j][7] * inv) << 16;
                    *reinterpret_cast<uint2 *>(q + (size_t)i * 8) = v;
                }
            }
        }
        parity ^= 1;
    }
}

// ---- the gradient ----------------------------------------------------------------

// The sums over the tokens a block keeps: dy * z * r2, and db * n, out of which both d_post (times the gate) and d_gate
// (times post) come where the gate is the same for all of the block's rows; else du * n.
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

template <int V, int kThreads, int kBlocks, bool kPost>
__global__ void __launch_bounds__(kThreads, kBlocks) block_norm_grad_kernel(const BlockNormArgs a, bool per_rank) {
    extern __shared__ __align__(16) float acc[];  // [sum][half of a vector][vector][4]
    __shared__ float part[3][2][2][kMaxWarps];
    const int H = a.g.H, nvec = H / 8, tid = threadIdx.x, width = blockDim.x;
    const bool branch = sum_branch(a);
    float4 *const acc4 = reinterpret_cast<float4 *>(acc);
    for (int i = tid; i < nvec; i += width)
        for (int q = 0; q < 2 * kSums; ++q) acc4[q * nvec + i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](int q, int i, const float (&f)[8]) {
        float4 &lo = acc4[(q * 2) * nvec + i], &hi = acc4[(q * 2 + 1) * nvec + i];
        float4 l = lo, h = hi;
        l.x += f[0], l.y += f[1], l.z += f[2], l.w += f[3];
        h.x += f[4], h.y += f[5], h.z += f[6], h.w += f[7];
        lo = l;
        hi = h;
    };
    long long row, end;
    block_rows(a.g, per_rank, gridDim.x, blockIdx.x, row, end);
    grid_dependency_wait();
    int parity = 0;
    const float inv_h = 1.0f / (float)H;
    const bool shared_gate = a.gate_kind != A2AV_GATE_TOKEN && (a.gate_kind != A2AV_GATE_RANK || per_rank);
    for (; row < end; ++row) {
        if (!row_active(a, row)) continue;
        const size_t at = (size_t)row * H;
        const uint16_t *gate = a.gate ? gate_row(a, row) : nullptr;
        const uint4 none = make_uint4(0, 0, 0, 0);
        uint4 xv[V], dyv[V], drv[V];
        float z[V][8];
        float sum = 0.0f, unused = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            const bool in = i < nvec;
            xv[j] = in ? ld_row(a.x + at + (size_t)i * 8) : none;
            unpack8(in ? ld_row(a.residual + at + (size_t)i * 8) : none, z[j]);
            dyv[j] = in && a.d_y ? ld_row(a.d_y + at + (size_t)i * 8) : none;
            drv[j] = in && a.d_residual_out ? ld_row(a.d_residual_out + at + (size_t)i * 8) : none;
        }
        if (row + 1 < end && tid < 4) {  // the next row on its way into L2
            const uint16_t *from = tid == 0 ? a.x : tid == 1 ? a.residual : tid == 2 ? a.d_y : a.d_residual_out;
            if (from) prefetch_row(from + at + H, 2 * H);
        }
        float r1 = 1.0f;
        if (kPost) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float x[8];
                unpack8(xv[j], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
            }
            block_reduce<false>(sum, unused, part[0][parity]);
            r1 = 1.0f / sqrtf(sum * inv_h + a.eps);
        }
        float zz = 0.0f, vz = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) continue;
            float u[8], w[8];
            unpack8(xv[j], u);
            if (kPost) {
                unpack8(ld_weight(a.post, i), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = u[e] * r1 * w[e];
            }
            if (gate) {
                unpack8(ld_weight(gate, i), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[j][e] = fmaf(a.branch_scale, u[e], a.residual_scale * z[j][e]);
                zz = fmaf(z[j][e], z[j][e], zz);
            }
            if (a.d_y) {
                float dy[8];
                unpack8(ld_weight(a.weight, i), w);
                unpack8(dyv[j], dy);
#pragma unroll
                for (int e = 0; e < 8; ++e) vz = fmaf(dy[e] * w[e], z[j][e], vz);
            }
        }
        float r2 = 0.0f, c2 = 0.0f;
        if (a.d_y) {
            block_reduce<false>(zz, vz, part[1][parity]);
            r2 = 1.0f / sqrtf(zz * inv_h + a.eps);
            c2 = r2 * r2 * r2 * (vz * inv_h);
        }
        float nx = 0.0f;
        float(&dn)[V][8] = z;  // z's place takes b * dz, then dn
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) continue;
            float dz[8], n[8], w[8];
            unpack8(drv[j], dz);
            if (a.d_y) {
                float dy[8];
                unpack8(dyv[j], dy);
                if (a.d_weight) {
                    float t[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] = dy[e] * (z[j][e] * r2);
                    add(kSumWeight, i, t);
                }
                unpack8(ld_weight(a.weight, i), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) dz[e] = fmaf(-c2, z[j][e], fmaf(dy[e] * w[e], r2, dz[e]));
            }
            {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = a.residual_scale * dz[e];
                st_v4(a.d_residual + at + (size_t)i * 8, pack8(t));
            }
            unpack8(xv[j], n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (kPost) n[e] *= r1;
                dn[j][e] = a.branch_scale * dz[e];
            }
            if (branch && shared_gate) {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = dn[j][e] * n[e];
                add(kSumBranch, i, t);
            }
            if (kPost) unpack8(ld_weight(a.post, i), w);
            if (a.d_gate && a.gate_kind == A2AV_GATE_TOKEN) {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = dn[j][e] * (kPost ? n[e] * w[e] : n[e]);
                st_v4(static_cast<uint16_t *>(a.d_gate) + at + (size_t)i * 8, pack8(t));
            }
            if (gate) {
                float gt[8];
                unpack8(ld_weight(gate, i), gt);
#pragma unroll
                for (int e = 0; e < 8; ++e) dn[j][e] *= gt[e];
            }
            if (kPost) {
                if (branch && !shared_gate) {
                    float t[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] = dn[j][e] * n[e];
                    add(kSumBranch, i, t);
                }
                float x[8];
                unpack8(xv[j], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dn[j][e] *= w[e];
                    nx = fmaf(dn[j][e], x[e], nx);
                }
            }
        }
        float c1 = 0.0f;
        if (kPost) {
            block_reduce<false>(nx, unused, part[2][parity]);
            c1 = r1 * r1 * r1 * (nx * inv_h);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) continue;
            float x[8];
            unpack8(xv[j], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(dn[j][e], r1, -(x[e] * c1));
            st_v4(a.d_x + at + (size_t)i * 8, pack8(x));
        }
        parity ^= 1;
    }
    for (int q = 0; q < kSums; ++q)
        if (q == kSumWeight ? a.d_weight != nullptr : branch)
            for (int i = tid; i < nvec; i += width) {
                float4 *out = reinterpret_cast<float4 *>(a.scratch + ((size_t)blockIdx.x * kSums + q) * H) + 2 * i;
                out[0] = acc4[(q * 2) * nvec + i];
                out[1] = acc4[(q * 2 + 1) * nvec + i];
            }
}

// The blocks' sums S added up: d_weight = sum S, d_post = sum gate * S, d_gate = post * sum S (per rank over its blocks).
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
        reinterpret_cast<float4 *>(out + (size_t)rank * H)[i] = s;
    }
}

int row_threads(int H, int V) { return ((H / 8 + V - 1) / V + 31) / 32 * 32; }

// Whether the gradient's blocks keep to a rank each.
bool keeps_to_rank(const BlockNormArgs &a) {
    return a.gate_kind == A2AV_GATE_RANK && (a.d_gate || a.d_post);
}

// Blocks of the gradient: what an SM holds, at most one per row, a multiple of R where each is to keep to a rank.
int grad_blocks(int num_sms, const Geometry &g, bool per_rank) {
    const int threads = row_threads(g.H, kV);
    const int per_sm = threads > 512 ? 1 : 1024 / threads < 16 ? 1024 / threads : 16;
    const long long rows = (long long)g.R * g.T, most = (long long)num_sms * per_sm;
    if (!per_rank) return (int)(rows < most ? rows : most);
    const long long parts = most / g.R < 1 ? 1 : most / g.R;
    return g.R * (int)(g.T < parts ? g.T : parts);
}

template <int V, int kThreads, int kBlocks, bool kPost>
cudaError_t launch_grad(const a2av_plan_s &p, const BlockNormArgs &a, int blocks, bool per_rank, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = block_norm_grad_kernel<V, kThreads, kBlocks, kPost>;
    const cudaError_t e =
        allow_smem(kernel, done, p.cfg.device, (size_t)kMaxNormGradRow * kSums * sizeof(float));
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, blocks, row_threads(a.g.H, V), (size_t)a.g.H * kSums * sizeof(float), s, a, per_rank);
}

template <bool kPost>
cudaError_t launch_norm_rows(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    const long long rows = (long long)a.g.R * a.g.T;
    const int H = a.g.H, threads = row_threads(H, H > 16384 ? 4 : kV);
    const long long per_sm = threads > 512 ? 1 : 1024 / threads < 16 ? 1024 / threads : 16;
    const long long cap = p.num_sms * per_sm;
    const int grid = (int)(rows < cap ? rows : cap);
    if (H > 16384) return launch_pdl(block_norm_kernel<4, 1024, 1, kPost>, grid, threads, 0, s, a);
    if (H > 8192) return launch_pdl(block_norm_kernel<kV, 1024, 1, kPost>, grid, threads, 0, s, a);
    return launch_pdl(block_norm_kernel<kV, 512, 2, kPost>, grid, threads, 0, s, a);
}

}  // namespace

cudaError_t launch_block_norm(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    return a.post ? launch_norm_rows<true>(p, a, s) : launch_norm_rows<false>(p, a, s);
}

int64_t norm_scratch_bytes(const a2av_plan_s &p) {
    const int one = grad_blocks(p.num_sms, p.g, false), ranks = grad_blocks(p.num_sms, p.g, true);
    return (int64_t)(one > ranks ? one : ranks) * kSums * p.g.H * (int64_t)sizeof(float);
}

cudaError_t launch_block_norm_grad(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s, int64_t &launches) {
    const bool per_rank = keeps_to_rank(a);
    const bool sums = a.d_weight || a.d_post || (a.d_gate && a.gate_kind != A2AV_GATE_TOKEN);
    const int blocks = grad_blocks(p.num_sms, a.g, per_rank);
    cudaError_t e = a.g.H > 8192 ? (a.post ? launch_grad<kV, 1024, 1, true>(p, a, blocks, per_rank, s)
                                           : launch_grad<kV, 1024, 1, false>(p, a, blocks, per_rank, s))
                                 : (a.post ? launch_grad<kV, 512, 2, true>(p, a, blocks, per_rank, s)
                                           : launch_grad<kV, 512, 2, false>(p, a, blocks, per_rank, s));
    if (e != cudaSuccess) return e;
    ++launches;
    if (!sums) return cudaSuccess;
    BlockNormArgs b = a;
    if (a.gate_kind == A2AV_GATE_TOKEN) b.d_gate = nullptr;
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
