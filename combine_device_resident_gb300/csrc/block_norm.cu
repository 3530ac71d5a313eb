// The norms before and after a block with its gate and the residual's scale,
// and their gradient.
//
//   u = x * r1 * post,            r1 = 1 / sqrt(mean x^2 + eps)
//   z = a * residual + b * gate * u,   residual_out = bf16(z)
//   v = z * weight * r2,          r2 = 1 / sqrt(mean z^2 + eps)
//
// post, gate and b are one factor per channel, in fp32 in shared memory, so z = (x * r1) * factor + a * residual.
// One block per row, the row in registers between its uses, the next one's loads on their way: every tensor is read once.
// Bound by HBM: 65,536 x 7168 583 us (6.44 TB/s).
//
// Gradient, dy and dr those of v and of residual_out, n = x * r1:
//   dv = dy * weight;  dz = dr + r2 * dv - z * (r2^3 * mean(dv z));  d_residual = a * dz
//   d_gate = b * dz * n * post;  dn = dz * factor;  dx = r1 * dn - x * (r1^3 * mean(dn x))
//   d_weight = sum dy * z * r2,  d_post = b * sum dz * gate * n   over the tokens
// z and the roots are taken again from x and residual: three block sums, each
// after the one before.  A block takes consecutive rows, two at a time; its threads keep their
// columns, so the sums over the tokens are each thread's own in shared memory;
// the blocks' sums are added by a second kernel in a fixed order.  65,536 x 7168: 1066 us (5.29 TB/s); bound by the way
// through a pair of rows: one block of 14 warps is on an SM, and 58% of its issue slots are empty.
#include "block_ops.cuh"
#include "expert_common.cuh"
#include "row_math.cuh"

namespace a2av {
namespace {

// Warps of a block's row, as block_sum counts them.
constexpr int warps_of(int threads) { return threads <= 512 ? 16 : 32; }

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
// Brings `bytes` (a multiple of 16) into L2.
__device__ __forceinline__ void prefetch_row(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Sums of N values over the block, of which every thread gets all.  With two a warp's halves take one each, with four its
// quarters, so that they cost little more than one.  `part` holds zeros where there is no warp, and is free again after the next barrier.
template <int N, int W>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*part)[W]) {
    static_assert((N == 1 || N == 2 || N == 4) && (W == 16 || (W == 32 && N < 4)), "values, warps");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kLanes = 32 / N;  // that carry a value: lane / kLanes names it
    float s = v[0];
    const bool up = lane & 16, odd = lane & 8;
    if constexpr (N == 2) s = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
    if constexpr (N == 4) {
        const float b0 = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
        const float b1 = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
        s = (odd ? b1 : b0) + __shfl_xor_sync(0xffffffffu, odd ? b0 : b1, 8);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((lane & (kLanes - 1)) == 0) part[lane / kLanes][warp] = s;
    __syncthreads();
    // a lane reads four warps' sums
    const float4 p = reinterpret_cast<const float4 *>(part[lane / kLanes])[lane & (W / 4 - 1)];
    s = (p.x + p.y) + (p.z + p.w);
#pragma unroll
    for (int o = W / 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = N == 1 ? s : __shfl_sync(0xffffffffu, s, n * kLanes);
}
// Zeros for block_sum; ends in a barrier.
template <int n>
__device__ __forceinline__ void clear_parts(float (&part)[n]) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) part[i] = 0.0f;
    __syncthreads();
}

// Largest magnitude of a warp's values, NaN if there is one.
__device__ __forceinline__ float warp_peak(float v) {
    float d;
    asm("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}

// A thread takes 16 consecutive values of a row (C times, the threads' width apart): 32 bytes of bf16 in one access where
// every row starts on 32 bytes (k32), else in two of 16, of which the row's last thread may have the first alone.
struct Bits {
    uint4 v[2];
};
template <bool k32>
__device__ __forceinline__ Bits ld16(const uint16_t *p, int left) {
    Bits b;
    if (k32) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(b.v[0].x), "=r"(b.v[0].y), "=r"(b.v[0].z), "=r"(b.v[0].w), "=r"(b.v[1].x), "=r"(b.v[1].y),
                       "=r"(b.v[1].z), "=r"(b.v[1].w)
                     : "l"(p)
                     : "memory");
    } else {
        b.v[0] = ld_row(p);
        b.v[1] = left > 8 ? ld_row(p + 8) : make_uint4(0, 0, 0, 0);
    }
    return b;
}
template <bool k32>
__device__ __forceinline__ void st16(uint16_t *p, int left, const uint4 &lo, const uint4 &hi) {
    if (k32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                     "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                     : "memory");
    } else {
        st_v4(p, lo);
        if (left > 8) st_v4(p + 8, hi);
    }
}
// A weight: the same for every row, so it stays in the L1 cache.
__device__ __forceinline__ Bits ld_weight(const uint16_t *w, int left) {
    Bits b;
    b.v[0] = __ldg(reinterpret_cast<const uint4 *>(w));
    b.v[1] = left > 8 ? __ldg(reinterpret_cast<const uint4 *>(w) + 1) : make_uint4(0, 0, 0, 0);
    return b;
}
__device__ __forceinline__ void unpack16(const Bits &b, pair (&f)[8]) {
    const uint32_t w[8] = {b.v[0].x, b.v[0].y, b.v[0].z, b.v[0].w, b.v[1].x, b.v[1].y, b.v[1].z, b.v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = both(lo_f(w[i]), hi_f(w[i]));
}
// Makes the compiler unpack these anew where they are used next: held unpacked over a block's sum they would cost twice
// the registers.
__device__ __forceinline__ void keep_packed(Bits &b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) asm volatile("" : "+r"(b.v[i].x), "+r"(b.v[i].y), "+r"(b.v[i].z), "+r"(b.v[i].w));
}
// Four of them.
__device__ __forceinline__ void unpack4(const Bits &b, int q, pair (&f)[2]) {
    const uint4 &v = b.v[q / 2];
    const uint32_t lo = q % 2 ? v.z : v.x, hi = q % 2 ? v.w : v.y;
    f[0] = both(lo_f(lo), hi_f(lo));
    f[1] = both(lo_f(hi), hi_f(hi));
}
__device__ __forceinline__ void scale4(pair (&f)[2], const Bits &b, int q) {
    pair g[2];
    unpack4(b, q, g);
    f[0] = mul2(f[0], g[0]);
    f[1] = mul2(f[1], g[1]);
}
template <bool k32>
__device__ __forceinline__ void store16(uint16_t *p, int left, const pair (&f)[8]) {
    st16<k32>(p, left, make_uint4(bf16_of(f[0]), bf16_of(f[1]), bf16_of(f[2]), bf16_of(f[3])),
              make_uint4(bf16_of(f[4]), bf16_of(f[5]), bf16_of(f[6]), bf16_of(f[7])));
}
constexpr int kEach = 16;  // values of a row per thread (and C)

// A row of fp32 in shared memory, [quarter of a thread's values][thread], so that a warp's 16-byte accesses lie side by
// side.  A thread touches its own columns alone.
__device__ __forceinline__ void ld_shared(const ulonglong2 *row, int slots, pair (&f)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const ulonglong2 v = row[q * slots];
        f[2 * q] = v.x, f[2 * q + 1] = v.y;
    }
}
__device__ __forceinline__ void st_shared(ulonglong2 *row, int slots, const pair (&f)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q * slots] = make_ulonglong2(f[2 * q], f[2 * q + 1]);
}

__device__ __forceinline__ void ld_quarter(const ulonglong2 *row, int slots, int q, pair (&f)[2]) {
    const ulonglong2 v = row[q * slots];
    f[0] = v.x, f[1] = v.y;
}
__device__ __forceinline__ void st_quarter(ulonglong2 *row, int slots, int q, const pair (&f)[2]) {
    row[q * slots] = make_ulonglong2(f[0], f[1]);
}

// The factor of x * r1 in z, per channel: branch_scale * post * gate, the gate left out where it is the token's own
// (gate null here).
template <int C>
__device__ __forceinline__ void set_coef(const BlockNormArgs &a, const uint16_t *gate, ulonglong2 *coef, int slots) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (threadIdx.x + c * blockDim.x) * kEach, left = a.g.H - at;
        if (left <= 0) continue;
        pair f[8], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = both(a.branch_scale);
        if (a.post) {
            unpack16(ld_weight(a.post + at, left), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = mul2(f[e], w[e]);
        }
        if (gate) {
            unpack16(ld_weight(gate + at, left), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = mul2(f[e], w[e]);
        }
        st_shared(coef + c * blockDim.x, slots, f);
    }
}

// The next row's loads are in registers while a row is worked on.  Rows of up to 8192 in blocks of up to 512 threads, two
// or more an SM (64 registers); to 16,384 in one of 1,024; beyond that 32 values a thread, of which some spill.
template <int C, int kThreads, int kBlocks, bool kPost, bool kToken, bool k32>
__global__ void __launch_bounds__(kThreads, kBlocks) block_norm_kernel(const BlockNormArgs a) {
    extern __shared__ __align__(16) ulonglong2 smem[];
    constexpr int W = warps_of(kThreads);
    __shared__ __align__(16) float parts[2 * 2 * 2 * W];
    auto part = reinterpret_cast<float(*)[2][2][W]>(parts);  // [which sum][row parity]
    clear_parts(parts);
    const int H = a.g.H, width = blockDim.x, slots = C * width;
    ulonglong2 *const coef = smem + threadIdx.x;
    const long long rows = (long long)a.g.R * a.g.T;
    const float inv_h = 1.0f / (float)H;
    const pair alpha = both(a.residual_scale);
    grid_dependency_wait();
    int parity = 0;
    Bits xv[C], rv[C], gv[C];
#pragma unroll
    for (int c = 0; c < C; ++c) xv[c] = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};  // behind the row's end
    long long row = blockIdx.x;
    auto load = [&] {  // from the first row on that takes part
        while (row < rows && !row_active(a, row)) row += gridDim.x;
        if (row >= rows) return;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (threadIdx.x + c * width) * kEach, left = H - col;
            const size_t at = (size_t)row * H + col;
            if (left <= 0) continue;
            xv[c] = ld16<k32>(a.x + at, left);
            rv[c] = ld16<k32>(a.residual + at, left);
            if (kToken) gv[c] = ld16<k32>(a.gate + at, left);
        }
    };
    load();
    const uint16_t *coef_of = nullptr;
    if (row < rows) set_coef<C>(a, coef_of = kToken || !a.gate ? nullptr : gate_row(a, row), coef, slots);
    while (row < rows) {
        const size_t base = (size_t)row * H;
        if (!kToken && a.gate_kind == A2AV_GATE_RANK && gate_row(a, row) != coef_of)
            set_coef<C>(a, coef_of = gate_row(a, row), coef, slots);
        uint8_t *q = a.rows8 ? a.rows8 + (size_t)row * (H + 16) : nullptr;
        pair z[C][8];
        float r1 = 1.0f, peak = 0.0f;
        if (kPost) {
            pair s = both(0.0f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                pair x[8];
                unpack16(xv[c], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fma2(x[e], x[e], s);
            }
            float sum[1] = {sum2(s)};
            block_sum<1, W>(sum, part[0][parity]);
            r1 = rsqrtf(fmaf(sum[0], inv_h, a.eps));
        }
        pair s = both(0.0f);
        const pair root = both(r1);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (threadIdx.x + c * width) * kEach, left = H - col;
            if (left <= 0) continue;
            pair x[8], f[8];
            unpack16(xv[c], x);
            unpack16(rv[c], z[c]);
            ld_shared(coef + c * width, slots, f);
            if (kToken) {
                pair g[8];
                unpack16(gv[c], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = mul2(f[e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[c][e] = fma2(kPost ? mul2(x[e], root) : x[e], f[e], mul2(z[c][e], alpha));
                s = fma2(z[c][e], z[c][e], s);
            }
            if (a.residual_out) store16<k32>(a.residual_out + base + col, left, z[c]);
            if (a.weight) {
                pair w[8];
                unpack16(ld_weight(a.weight + col, left), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[c][e] = mul2(z[c][e], w[e]);
                if (a.rows8)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float lo, hi;
                        split(z[c][e], lo, hi);
                        peak = max_nan(peak, max_nan(fabsf(lo), fabsf(hi)));
                    }
            }
        }
        row += gridDim.x;
        load();
        if (a.weight) {
            const int lane = threadIdx.x & 31;
            float *const peaks = part[1][parity][1];
            if (a.rows8) {
                peak = warp_peak(peak);
                if (lane == 0) peaks[threadIdx.x >> 5] = peak;
            }
            float sum[1] = {sum2(s)};
            block_sum<1, W>(sum, part[1][parity]);  // its barrier is the peaks', too
            const float r2 = rsqrtf(fmaf(sum[0], inv_h, a.eps));
            const pair root2 = both(r2);
            float inv = 0.0f;
            if (a.rows8) {
                peak = warp_peak(lane < (width >> 5) ? peaks[lane] : 0.0f) * r2;
                const bool zero = peak < kZeroRow;  // false for NaN
                inv = zero ? 0.0f : kLow8 / peak;
                if (threadIdx.x == 0) st_v4(q + H, make_uint4(__float_as_uint(zero ? 0.0f : peak / kLow8), 0, 0, 0));
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (threadIdx.x + c * width) * kEach, left = H - col;
                if (left <= 0) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) z[c][e] = mul2(z[c][e], root2);
                if (a.y) store16<k32>(a.y + base + col, left, z[c]);
                if (q) {  // H is a multiple of 16
                    uint32_t b[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float lo, hi;
                        split(mul2(z[c][e], both(inv)), lo, hi);
                        b[e] = e4m3x2(lo, hi);
                    }
                    st_v4(q + col, make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16));
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

// Rows of block b: consecutive, and of one rank where the gate is per rank.
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

template <bool kPost, bool kToken, bool k32>
__global__ void __launch_bounds__(1024, 1) block_norm_grad_kernel(const BlockNormArgs a, bool per_rank) {
    extern __shared__ __align__(16) ulonglong2 smem[];
    constexpr int W = 32;
    __shared__ __align__(16) float parts[3 * 2 * 2 * W];
    auto part = reinterpret_cast<float(*)[2][2][W]>(parts);  // [which sum][row parity]
    clear_parts(parts);
    const int H = a.g.H, width = blockDim.x;
    const bool branch = sum_branch(a), in = (int)threadIdx.x * kEach < H;
    // a thread behind the row's end loads what the first one does and takes no part in sums and stores
    const int col = in ? threadIdx.x * kEach : 0, left = H - col;
    ulonglong2 *const coef = smem + threadIdx.x;
    ulonglong2 *const acc[kSums] = {coef + 4 * width, coef + 8 * width};
    {
        const pair zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int q = 0; q < kSums; ++q) st_shared(acc[q], width, zero);
    }
    long long row, end;
    block_rows(a.g, per_rank, gridDim.x, blockIdx.x, row, end);
    grid_dependency_wait();
    int parity = 0;
    const float inv_h = 1.0f / (float)H;
    const pair alpha = both(a.residual_scale);
    if (row < end) set_coef<1>(a, kToken || !a.gate ? nullptr : gate_row(a, row), coef, width);
    const uint16_t *const weight = a.weight + col;
    for (; row < end; ++row) {
        if (!row_active(a, row)) continue;
        const size_t at = (size_t)row * H + col;
        Bits xv, rv, dyv, drv, gv;
        xv = ld16<k32>(a.x + at, left);
        rv = ld16<k32>(a.residual + at, left);
        if (a.d_y) dyv = ld16<k32>(a.d_y + at, left);
        if (a.d_residual_out) drv = ld16<k32>(a.d_residual_out + at, left);
        else drv = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};
        if (kToken) gv = ld16<k32>(a.gate + at, left);
        if (row + 1 < end && threadIdx.x < 5) {  // the next row on its way into L2
            const int t = threadIdx.x;
            const uint16_t *from = t == 0   ? a.x
                                   : t == 1 ? a.residual
                                   : t == 2 ? a.d_y
                                   : t == 3 ? a.d_residual_out
                                   : kToken ? a.gate
                                            : nullptr;
            if (from) prefetch_row(from + (size_t)(row + 1) * H, 2 * H);
        }
        float r1 = 1.0f;
        if (kPost) {
            pair x[8], s = both(0.0f);
            unpack16(xv, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fma2(x[e], x[e], s);
            float sum[1] = {in ? sum2(s) : 0.0f};
            block_sum<1, W>(sum, part[0][parity]);
            r1 = rsqrtf(fmaf(sum[0], inv_h, a.eps));
            keep_packed(xv);
        }
        const pair root1 = both(r1);
        pair z[8], zz = both(0.0f), vz = both(0.0f);
        {
            Bits wv;
            if (a.d_y) wv = ld_weight(weight, left);
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // four values at a time: what they need is soon free again
                pair x[2], f[2], r[2], dy[2], w[2];
                unpack4(xv, q, x);
                unpack4(rv, q, r);
                ld_quarter(coef, width, q, f);
                if (kToken) scale4(f, gv, q);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    z[2 * q + e] = fma2(kPost ? mul2(x[e], root1) : x[e], f[e], mul2(r[e], alpha));
                    zz = fma2(z[2 * q + e], z[2 * q + e], zz);
                }
                if (a.d_y) {
                    unpack4(wv, q, w);
                    unpack4(dyv, q, dy);
#pragma unroll
                    for (int e = 0; e < 2; ++e) vz = fma2(mul2(dy[e], w[e]), z[2 * q + e], vz);
                }
            }
        }
        float r2 = 0.0f, c2 = 0.0f;
        if (a.d_y) {
            float sum[2] = {in ? sum2(zz) : 0.0f, in ? sum2(vz) : 0.0f};
            block_sum<2, W>(sum, part[1][parity]);
            r2 = rsqrtf(fmaf(sum[0], inv_h, a.eps));
            c2 = r2 * (r2 * (r2 * (sum[1] * inv_h)));  // the cube alone may overflow
            keep_packed(xv);
            keep_packed(dyv);
            if (kToken) keep_packed(gv);
        }
        pair nx = both(0.0f);
        pair(&dn)[8] = z;  // z's place takes dz * coef: the gradient of n = x * r1
        if (in) {
            const pair root2 = both(r2), less2 = both(-c2);
            Bits wv;
            uint32_t dr[8], dg[8];
            if (a.d_y) wv = ld_weight(weight, left);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                pair dz[2], x[2], n[2], f[2], t[2];
                unpack4(drv, q, dz);
                if (a.d_y) {
                    pair dy[2], w[2];
                    unpack4(dyv, q, dy);
                    unpack4(wv, q, w);
                    if (a.d_weight) {
                        ld_quarter(acc[kSumWeight], width, q, t);
#pragma unroll
                        for (int e = 0; e < 2; ++e) t[e] = fma2(dy[e], mul2(z[2 * q + e], root2), t[e]);
                        st_quarter(acc[kSumWeight], width, q, t);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) dz[e] = fma2(less2, z[2 * q + e], fma2(mul2(dy[e], w[e]), root2, dz[e]));
                }
                unpack4(xv, q, x);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    dr[2 * q + e] = bf16_of(mul2(dz[e], alpha));
                    n[e] = kPost ? mul2(x[e], root1) : x[e];
                }
                ld_quarter(coef, width, q, f);
                if (kToken) {  // b * dz * u
#pragma unroll
                    for (int e = 0; e < 2; ++e) dg[2 * q + e] = bf16_of(mul2(mul2(dz[e], f[e]), n[e]));
                    scale4(f, gv, q);
                }
                if (branch) {
                    pair d[2] = {dz[0], dz[1]};
                    if (kToken) scale4(d, gv, q);
                    ld_quarter(acc[kSumBranch], width, q, t);
#pragma unroll
                    for (int e = 0; e < 2; ++e) t[e] = fma2(d[e], n[e], t[e]);
                    st_quarter(acc[kSumBranch], width, q, t);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    dn[2 * q + e] = mul2(dz[e], f[e]);
                    if (kPost) nx = fma2(dn[2 * q + e], x[e], nx);
                }
            }
            st16<k32>(a.d_residual + at, left, make_uint4(dr[0], dr[1], dr[2], dr[3]), make_uint4(dr[4], dr[5], dr[6], dr[7]));
            if (kToken && a.d_gate)
                st16<k32>(static_cast<uint16_t *>(a.d_gate) + at, left, make_uint4(dg[0], dg[1], dg[2], dg[3]),
                          make_uint4(dg[4], dg[5], dg[6], dg[7]));
        }
        float c1 = 0.0f;
        if (kPost) {
            float sum[1] = {sum2(nx)};
            block_sum<1, W>(sum, part[2][parity]);
            c1 = r1 * (r1 * (r1 * (sum[0] * inv_h)));
            keep_packed(xv);
        }
        if (in) {
            if (kPost) {
                const pair less1 = both(-c1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    pair x[2];
                    unpack4(xv, q, x);
#pragma unroll
                    for (int e = 0; e < 2; ++e) dn[2 * q + e] = fma2(dn[2 * q + e], root1, mul2(x[e], less1));
                }
            }
            store16<k32>(a.d_x + at, left, dn);
        }
        parity ^= 1;
    }
    if (in)
        for (int q = 0; q < kSums; ++q)
            if (q == kSumWeight ? a.d_weight != nullptr : branch) {
                ulonglong2 *out =
                    reinterpret_cast<ulonglong2 *>(a.scratch + ((size_t)blockIdx.x * kSums + q) * H + col);
                for (int e = 0; e < (left > 8 ? 4 : 2); ++e) out[e] = acc[q][e * width];
            }
}

// Rows of up to 8192 two at a time: both rows' values are in registers, the factors, the weights in fp32
// and the sums over the tokens are read from shared memory once for both, and a block sum serves both.  That is half the
// shared-memory traffic and half the barriers of the form above, which takes the longer rows.  128 registers a thread, of
// which some values spill: 36 bytes a thread without the post norm, 144 with it, 550-690 with a gate per token (the form
// above: 84, 140, 280-300).  All the same it is the faster one at each width timed, in us against the form above, post
// norm and a gate per channel, then per token: 65,536 x 2048 279 (458), 439 (726); 2,040 x 5120 44 (57), 53 (75);
// 26,208 x 5120 358 (448), 490 (658); 16,384 x 7168 283 (412), 422 (595); 16,384 x 8192 318 (507), 475 (780).  Eight
// values a thread and twice the threads took 1355 on 65,536 x 7168.
template <bool kPost, bool kToken, bool k32>
__global__ void __launch_bounds__(512, 1) block_norm_grad_pair_kernel(const BlockNormArgs a, bool per_rank) {
    extern __shared__ __align__(16) ulonglong2 smem[];
    constexpr int W = 16;
    __shared__ __align__(16) float parts[2 * 3 * 4 * W];
    auto part = reinterpret_cast<float(*)[3][4][W]>(parts);  // [parity of the turn][which sum]
    clear_parts(parts);
    const int H = a.g.H, width = blockDim.x;
    const bool branch = sum_branch(a), in = (int)threadIdx.x * kEach < H;
    // a thread behind the row's end loads what the first one does and takes no part in sums and stores
    const int col = in ? threadIdx.x * kEach : 0, left = H - col;
    ulonglong2 *const coef = smem + threadIdx.x, *const weight = coef + 4 * width;
    ulonglong2 *const acc[kSums] = {coef + 8 * width, coef + 12 * width};
    {
        const pair zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int q = 0; q < kSums; ++q) st_shared(acc[q], width, zero);
    }
    long long next, end;
    block_rows(a.g, per_rank, gridDim.x, blockIdx.x, next, end);
    grid_dependency_wait();
    const float inv_h = 1.0f / (float)H;
    const pair alpha = both(a.residual_scale);
    if (next < end) set_coef<1>(a, kToken || !a.gate ? nullptr : gate_row(a, next), coef, width);
    if (a.d_y) {
        pair w[8];
        unpack16(ld_weight(a.weight + col, left), w);
        st_shared(weight, width, w);
    }
    auto take = [&] {  // the next row that takes part, or -1
        while (next < end && !row_active(a, next)) ++next;
        return next < end ? next++ : -1;
    };
    for (int parity = 0;; parity ^= 1) {
        const long long row0 = take(), row1 = row0 < 0 ? -1 : take();
        if (row0 < 0) break;
        const bool two = row1 >= 0;  // else the first one's values stand in for the second's, and go nowhere
        const size_t at[2] = {(size_t)row0 * H + col, (size_t)(two ? row1 : row0) * H + col};
        Bits xv[2], rv[2], dyv[2], drv[2], gv[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            xv[r] = ld16<k32>(a.x + at[r], left);
            rv[r] = ld16<k32>(a.residual + at[r], left);
            if (a.d_y) dyv[r] = ld16<k32>(a.d_y + at[r], left);
            if (a.d_residual_out) drv[r] = ld16<k32>(a.d_residual_out + at[r], left);
            else drv[r] = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};
            if (kToken) gv[r] = ld16<k32>(a.gate + at[r], left);
        }
        if (next < end && threadIdx.x < 5) {  // the next two rows on their way into L2
            const int t = threadIdx.x;
            const uint16_t *from = t == 0   ? a.x
                                   : t == 1 ? a.residual
                                   : t == 2 ? a.d_y
                                   : t == 3 ? a.d_residual_out
                                   : kToken ? a.gate
                                            : nullptr;
            if (from) prefetch_row(from + (size_t)next * H, (next + 1 < end ? 4 : 2) * H);
        }
        float r1[2] = {1.0f, 1.0f};
        if (kPost) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                pair s = both(0.0f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    pair x[2];
                    unpack4(xv[r], q, x);
                    s = fma2(x[1], x[1], fma2(x[0], x[0], s));
                }
                r1[r] = in ? sum2(s) : 0.0f;
            }
            block_sum<2, W>(r1, part[parity][0]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                r1[r] = rsqrtf(fmaf(r1[r], inv_h, a.eps));
                keep_packed(xv[r]);
            }
        }
        pair z[2][8];
        float r2[2] = {0.0f, 0.0f}, c2[2] = {0.0f, 0.0f};
        {
            pair zz[2] = {0, 0}, vz[2] = {0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                pair f[2], w[2];
                ld_quarter(coef, width, q, f);
                if (a.d_y) ld_quarter(weight, width, q, w);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    pair x[2], y[2], dy[2], c[2] = {f[0], f[1]};
                    unpack4(xv[r], q, x);
                    unpack4(rv[r], q, y);
                    if (kToken) scale4(c, gv[r], q);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        pair &to = z[r][2 * q + e];
                        to = fma2(kPost ? mul2(x[e], both(r1[r])) : x[e], c[e], mul2(y[e], alpha));
                        zz[r] = fma2(to, to, zz[r]);
                    }
                    if (a.d_y) {
                        unpack4(dyv[r], q, dy);
#pragma unroll
                        for (int e = 0; e < 2; ++e) vz[r] = fma2(mul2(dy[e], w[e]), z[r][2 * q + e], vz[r]);
                    }
                }
            }
            if (a.d_y) {
                float sum[4] = {in ? sum2(zz[0]) : 0.0f, in ? sum2(zz[1]) : 0.0f, in ? sum2(vz[0]) : 0.0f,
                                in ? sum2(vz[1]) : 0.0f};
                block_sum<4, W>(sum, part[parity][1]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    r2[r] = rsqrtf(fmaf(sum[r], inv_h, a.eps));
                    c2[r] = r2[r] * (r2[r] * (r2[r] * (sum[2 + r] * inv_h)));  // the cube alone may overflow
                    keep_packed(xv[r]);
                    keep_packed(dyv[r]);
                    if (kToken) keep_packed(gv[r]);
                }
            }
        }
        pair nx[2] = {0, 0};
        if (in) {
            uint32_t dr[2][8], dg[2][8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                pair f[2], w[2], t[2], b[2];
                ld_quarter(coef, width, q, f);
                if (a.d_y) ld_quarter(weight, width, q, w);
                if (a.d_weight) ld_quarter(acc[kSumWeight], width, q, t);
                if (branch) ld_quarter(acc[kSumBranch], width, q, b);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    pair dz[2], x[2], n[2], c[2] = {f[0], f[1]};
                    unpack4(drv[r], q, dz);
                    if (a.d_y) {
                        pair dy[2];
                        unpack4(dyv[r], q, dy);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const pair zr = mul2(z[r][2 * q + e], both(r2[r]));
                            if (a.d_weight && (r == 0 || two)) t[e] = fma2(dy[e], zr, t[e]);
                            dz[e] = fma2(both(-c2[r]), z[r][2 * q + e], fma2(mul2(dy[e], w[e]), both(r2[r]), dz[e]));
                        }
                    }
                    unpack4(xv[r], q, x);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        dr[r][2 * q + e] = bf16_of(mul2(dz[e], alpha));
                        n[e] = kPost ? mul2(x[e], both(r1[r])) : x[e];
                    }
                    if (kToken) {  // b * dz * u
#pragma unroll
                        for (int e = 0; e < 2; ++e) dg[r][2 * q + e] = bf16_of(mul2(mul2(dz[e], c[e]), n[e]));
                        scale4(c, gv[r], q);
                    }
                    if (branch && (r == 0 || two)) {
                        pair d[2] = {dz[0], dz[1]};
                        if (kToken) scale4(d, gv[r], q);
#pragma unroll
                        for (int e = 0; e < 2; ++e) b[e] = fma2(d[e], n[e], b[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        pair &dn = z[r][2 * q + e];  // in z's place: the gradient of n = x * r1
                        dn = mul2(dz[e], c[e]);
                        if (kPost) nx[r] = fma2(dn, x[e], nx[r]);
                    }
                }
                if (a.d_weight) st_quarter(acc[kSumWeight], width, q, t);
                if (branch) st_quarter(acc[kSumBranch], width, q, b);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (r == 0 || two) {
                    st16<k32>(a.d_residual + at[r], left, make_uint4(dr[r][0], dr[r][1], dr[r][2], dr[r][3]),
                              make_uint4(dr[r][4], dr[r][5], dr[r][6], dr[r][7]));
                    if (kToken && a.d_gate)
                        st16<k32>(static_cast<uint16_t *>(a.d_gate) + at[r], left,
                                  make_uint4(dg[r][0], dg[r][1], dg[r][2], dg[r][3]),
                                  make_uint4(dg[r][4], dg[r][5], dg[r][6], dg[r][7]));
                }
        }
        float c1[2] = {sum2(nx[0]), sum2(nx[1])};
        if (kPost) {
            block_sum<2, W>(c1, part[parity][2]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                c1[r] = r1[r] * (r1[r] * (r1[r] * (c1[r] * inv_h)));
                keep_packed(xv[r]);
            }
        }
        if (in)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (kPost)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        pair x[2];
                        unpack4(xv[r], q, x);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            z[r][2 * q + e] = fma2(z[r][2 * q + e], both(r1[r]), mul2(x[e], both(-c1[r])));
                    }
                if (r == 0 || two) store16<k32>(a.d_x + at[r], left, z[r]);
            }
    }
    if (in)
        for (int q = 0; q < kSums; ++q)
            if (q == kSumWeight ? a.d_weight != nullptr : branch) {
                ulonglong2 *out =
                    reinterpret_cast<ulonglong2 *>(a.scratch + ((size_t)blockIdx.x * kSums + q) * H + col);
                for (int e = 0; e < (left > 8 ? 4 : 2); ++e) out[e] = acc[q][e * width];
            }
}

// The blocks' sums S added up: d_weight = sum S (blockIdx.y 0); S_r = sum S over the blocks of rank r (of all, without
// a gate per rank), d_gate[r] = b * post * S_r, d_post = b * sum_r gate[r] * S_r (blockIdx.y 1).  A block takes 32
// columns, eight threads in 32 groups: each group adds up a share of one rank's blocks, the shares and then the ranks are
// added in order.
constexpr int kSumGroups = 32;

__global__ void __launch_bounds__(8 * kSumGroups) norm_sums_kernel(const BlockNormArgs a, int blocks, bool per_rank) {
    __shared__ float4 part[kSumGroups][8], ranked[kSumGroups][8];
    const int H = a.g.H, x = threadIdx.x & 7, group = threadIdx.x >> 3, i = blockIdx.x * 8 + x;  // four columns
    const bool weights = blockIdx.y == 0, in = i < H / 4;
    float *const d_gate = static_cast<float *>(a.d_gate);
    const int R = per_rank && !weights ? a.g.R : 1, parts = blocks / R;
    const int share = R <= kSumGroups ? kSumGroups / R : 1, at_once = kSumGroups / share;  // groups per rank, ranks
    grid_dependency_wait();
    if (weights ? !a.d_weight : !a.d_post && !d_gate) return;
    auto add4 = [](float4 &s, const float4 &v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    auto times = [&](const float4 &s, const uint16_t *w) {
        const uint2 v = *(reinterpret_cast<const uint2 *>(w) + i);
        return make_float4(s.x * lo_f(v.x), s.y * hi_f(v.x), s.z * lo_f(v.y), s.w * hi_f(v.y));
    };
    auto store = [&](float *to, float4 s, float by) {
        s.x *= by, s.y *= by, s.z *= by, s.w *= by;
        reinterpret_cast<float4 *>(to)[i] = s;
    };
    // Whether any token of the sum took part: an empty one is zero, whatever the weights it would be multiplied by hold
    // (a rank without tokens may have no gate).
    auto has_tokens = [&](int r) {
        if (!a.num_tokens) return true;
        for (int s = per_rank ? r : 0; s < (per_rank ? r + 1 : a.g.R); ++s)
            if (active_tokens(a.num_tokens, s, a.g.T) > 0) return true;
        return false;
    };
    const float *const from = a.scratch + (size_t)(weights ? kSumWeight : kSumBranch) * H;
    float4 total = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int base = 0; base < R; base += at_once) {
        const int rank = base + group / share, mine = group % share;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in && group / share < at_once && rank < R) {
            const int first = rank * parts + (int)((long long)parts * mine / share);
            const int end = rank * parts + (int)((long long)parts * (mine + 1) / share);
#pragma unroll 4
            for (int b = first; b < end; ++b) add4(s, *(reinterpret_cast<const float4 *>(from + (size_t)b * kSums * H) + i));
        }
        part[group][x] = s;
        __syncthreads();
        if (in && group < at_once && base + group < R) {  // this thread: rank base + group
            const int r = base + group;
            float4 sum = part[group * share][x];
            for (int q = 1; q < share; ++q) add4(sum, part[group * share + q][x]);
            const bool live = !weights && has_tokens(r);
            if (!weights && d_gate) store(d_gate + (size_t)r * H, live && a.post ? times(sum, a.post) : sum, a.branch_scale);
            const bool shared_gate = a.gate_kind == A2AV_GATE_CHANNEL || a.gate_kind == A2AV_GATE_RANK;
            ranked[group][x] = live && shared_gate ? times(sum, a.gate + (size_t)r * H) : sum;
        }
        __syncthreads();
        if (in && group == 0)
            for (int q = 0; q < at_once && base + q < R; ++q) add4(total, ranked[q][x]);
    }
    if (in && group == 0 && (weights || a.d_post)) store(weights ? a.d_weight : a.d_post, total, weights ? 1.0f : a.branch_scale);
}

// Threads of a row, each with C times 16 values of it.
int row_threads(int H, int C = 1) { return ((H + kEach * C - 1) / (kEach * C) + 31) / 32 * 32; }

// Blocks of `threads` threads and `smem` bytes each that an SM holds, with `regs` registers a thread.
int blocks_per_sm(int threads, int regs, size_t smem) {
    const int by_regs = 65536 / (threads * regs), by_smem = (int)(228 * 1024 / (smem + 3 * 1024));
    const int n = by_regs < by_smem ? by_regs : by_smem;
    return n < 1 ? 1 : n > 32 ? 32 : n;
}
size_t coef_bytes(int H, int C = 1) { return (size_t)row_threads(H, C) * C * kEach * sizeof(float); }
constexpr int kPairRow = 8192;  // rows of the gradient's form that takes two at a time, at most
size_t grad_smem(int H) { return coef_bytes(H) * (1 + kSums + (H <= kPairRow)); }

// Blocks of the gradient: what the SMs hold, at most one per row, a multiple of R where each keeps to a rank.
int grad_blocks(int num_sms, const Geometry &g, bool per_rank) {
    const long long rows = (long long)g.R * g.T;
    const long long most =
        (long long)num_sms * blocks_per_sm(row_threads(g.H), g.H <= kPairRow ? 128 : 64, grad_smem(g.H));
    if (!per_rank) return (int)(rows < most ? rows : most);
    const long long parts = most / g.R < 1 ? 1 : most / g.R;
    return g.R * (int)(g.T < parts ? g.T : parts);
}

// Every row of every tensor on 32 bytes.
bool rows_on_32(const BlockNormArgs &a) {
    const void *const tensors[] = {a.x, a.residual, a.residual_out, a.y, a.d_y, a.d_residual_out, a.d_x, a.d_residual,
                                   a.gate_kind == A2AV_GATE_TOKEN ? a.gate : nullptr,
                                   a.gate_kind == A2AV_GATE_TOKEN ? a.d_gate : nullptr};
    uintptr_t bits = (uintptr_t)a.g.H * 2;
    for (const void *t : tensors) bits |= reinterpret_cast<uintptr_t>(t);
    return bits % 32 == 0;
}

template <int C, int kThreads, int kBlocks, bool kPost, bool kToken, bool k32>
cudaError_t launch_norm(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = block_norm_kernel<C, kThreads, kBlocks, kPost, kToken, k32>;
    const size_t smem = coef_bytes(a.g.H, C);
    const cudaError_t e = allow_smem(kernel, done, p.cfg.device, coef_bytes(kMaxNormRow, C));
    if (e != cudaSuccess) return e;
    const int threads = row_threads(a.g.H, C);
    const long long rows = (long long)a.g.R * a.g.T, cap = (long long)p.num_sms * blocks_per_sm(threads, 64, smem);
    return launch_pdl(kernel, (int)(rows < cap ? rows : cap), threads, smem, s, a);
}

template <bool kPost, bool kToken, bool k32>
cudaError_t launch_norm_rows(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    if (a.g.H > 16384) return launch_norm<2, 1024, 1, kPost, kToken, k32>(p, a, s);
    if (a.g.H > 8192) return launch_norm<1, 1024, 1, kPost, kToken, k32>(p, a, s);
    return launch_norm<1, 512, 2, kPost, kToken, k32>(p, a, s);
}

template <bool kPost, bool kToken, bool k32>
cudaError_t launch_grad_rows(const a2av_plan_s &p, const BlockNormArgs &a, int blocks, cudaStream_t s) {
    static std::atomic<uint64_t> done[2];
    const bool pairs = a.g.H <= kPairRow;
    const auto kernel =
        pairs ? block_norm_grad_pair_kernel<kPost, kToken, k32> : block_norm_grad_kernel<kPost, kToken, k32>;
    const cudaError_t e = allow_smem(kernel, done[pairs], p.cfg.device, grad_smem(pairs ? kPairRow : kMaxNormGradRow));
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, blocks, row_threads(a.g.H), grad_smem(a.g.H), s, a, a.gate_kind == A2AV_GATE_RANK);
}

// f<kPost, kToken, k32>, by what the call has.
#define A2AV_FORMS(f, ...)                                                                                     \
    (a.post ? (token ? (wide ? f<true, true, true>(__VA_ARGS__) : f<true, true, false>(__VA_ARGS__))           \
                     : (wide ? f<true, false, true>(__VA_ARGS__) : f<true, false, false>(__VA_ARGS__)))        \
            : (token ? (wide ? f<false, true, true>(__VA_ARGS__) : f<false, true, false>(__VA_ARGS__))         \
                     : (wide ? f<false, false, true>(__VA_ARGS__) : f<false, false, false>(__VA_ARGS__))))

}  // namespace

cudaError_t launch_block_norm(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s) {
    const bool token = a.gate_kind == A2AV_GATE_TOKEN, wide = rows_on_32(a);
    return A2AV_FORMS(launch_norm_rows, p, a, s);
}

int64_t norm_scratch_bytes(const a2av_plan_s &p) {
    const int one = grad_blocks(p.num_sms, p.g, false), ranks = grad_blocks(p.num_sms, p.g, true);
    return (int64_t)(one > ranks ? one : ranks) * kSums * p.g.H * (int64_t)sizeof(float);
}

cudaError_t launch_block_norm_grad(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s, int64_t &launches) {
    const bool token = a.gate_kind == A2AV_GATE_TOKEN, per_rank = a.gate_kind == A2AV_GATE_RANK, wide = rows_on_32(a);
    const bool sums = a.d_weight || a.d_post || (a.d_gate && !token);
    const int blocks = grad_blocks(p.num_sms, a.g, per_rank);
    cudaError_t e = A2AV_FORMS(launch_grad_rows, p, a, blocks, s);
    if (e != cudaSuccess) return e;
    ++launches;
    if (!sums) return cudaSuccess;
    BlockNormArgs b = a;
    if (token) b.d_gate = nullptr;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.g.H / 4 + 7) / 8, 2);
    cfg.blockDim = dim3(8 * kSumGroups);
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
