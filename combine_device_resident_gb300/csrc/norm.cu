// Root-mean-square norm with the residual's addition, in bf16 and/or as 8-bit
// rows with scales, and the 8-bit rows of an arena without the norm.
//
//   z = x + residual                       fp32, residual_out = bf16(z)
//   t_i = z_i * w_i,  r = 1 / sqrt(mean z^2 + eps),  v_i = t_i * r
//   y = bf16(v);  a = max|v|;  scale = a / 448;  q = e4m3(v * (448 / a))
//
// One block per row (short rows: one warp), the row in registers between the two uses of it, so x
// and the residual are read once.  Rounding is monotone, so max|v| is exactly
// max|t| * r: the sum of squares and the maximum come out of one block
// reduction and there is one barrier per row.  Bound by HBM: 2 + 2 bytes read,
// 2 + (1 or 2) written per element.
#include <cuda_bf16.h>

#include "a2av_internal.cuh"

namespace a2av {
namespace {

constexpr float kLow8 = 448.0f;      // largest finite e4m3
constexpr float kZeroRow = 1e-30f;   // a row whose maximum is below this is stored as zeros

// NaN-keeping maximum: a NaN anywhere in a row has to reach its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Rounded to nearest even, values past 448 (one rounding of 448/a away at most) to 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Row `row` of the token arrays takes part / row `row` of the arena is live.
template <bool kNorm>
__device__ __forceinline__ bool row_active(const NormArgs &a, int row) {
    if (kNorm) {
        if (!a.num_tokens) return true;
        const int s = row / a.g.T;
        return row - s * a.g.T < active_tokens(a.num_tokens, s, a.g.T);
    }
    if (a.g.window_mode == A2AV_WINDOW_FIXED) {
        const int d = (int)(row / a.g.window_rows);
        return row - (long long)d * a.g.window_rows < __ldg(a.recv_total + d);
    }
    return row < __ldg(a.window_base + a.g.R - 1) + __ldg(a.recv_total + a.g.R - 1);
}

// The first row from `row` on, in steps of `step`, that takes part; a.rows if none.
template <bool kNorm>
__device__ __forceinline__ int next_row(const NormArgs &a, long long row, int step) {
    while (row < a.rows && !row_active<kNorm>(a, (int)row)) row += step;
    return (int)min(row, (long long)a.rows);
}

// V 16-byte vectors of a row per thread; a block, or with kWarp each of its warps, takes a row at a time.
template <int V, int kThreads, int kBlocks, bool kNorm, bool kWarp>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_kernel(NormArgs a) {
    __shared__ float part[2][2][32];  // [row parity][sum, max][warp]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int tid = kWarp ? lane : threadIdx.x, width = kWarp ? 32 : blockDim.x;  // among the threads of the row
    const int step = kWarp ? gridDim.x * nwarps : gridDim.x;                      // rows in progress
    const int nvec = a.H >> 3;
    grid_dependency_wait();

    uint4 w[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = tid + j * width;
        w[j] = kNorm && i < nvec ? ld_stream_v4(a.weight + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
    }
    int parity = 0;
    uint4 xv[V], rv[V];
    int row = next_row<kNorm>(a, kWarp ? blockIdx.x * nwarps + warp : blockIdx.x, step);
    auto load = [&] {  // the next row is asked for while this one is finished
        if (row >= a.rows) return;
        const size_t at = (size_t)row * a.H;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            xv[j] = i < nvec ? ld_row(a.x + at + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
            rv[j] = kNorm && a.residual && i < nvec ? ld_row(a.residual + at + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
        }
    };
    load();
    while (row < a.rows) {
        const size_t at = (size_t)row * a.H;
        uint8_t *q = a.rows8 ? a.rows8 + (size_t)row * (a.H + 16) : nullptr;
        float t[V][8];
        float sum = 0.0f, peak = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            const uint32_t xs[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
            const uint32_t rs[4] = {rv[j].x, rv[j].y, rv[j].z, rv[j].w};
            const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
            uint32_t zs[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                float z0 = lo_f(xs[p]), z1 = hi_f(xs[p]);
                if (kNorm) {
                    z0 += lo_f(rs[p]);
                    z1 += hi_f(rs[p]);
                    sum = fmaf(z0, z0, sum);
                    sum = fmaf(z1, z1, sum);
                    zs[p] = bf16x2(z0, z1);
                    z0 *= lo_f(ws[p]);
                    z1 *= hi_f(ws[p]);
                }
                t[j][2 * p] = z0;
                t[j][2 * p + 1] = z1;
                peak = max_nan(peak, max_nan(fabsf(z0), fabsf(z1)));
            }
            if (kNorm && a.residual_out && i < nvec)
                st_v4(a.residual_out + at + (size_t)i * 8, make_uint4(zs[0], zs[1], zs[2], zs[3]));
        }
        row = next_row<kNorm>(a, (long long)row + step, step);
        load();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (kNorm) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            peak = max_nan(peak, __shfl_xor_sync(0xffffffffu, peak, o));
        }
        if (!kWarp) {
            if (lane == 0) {
                part[parity][0][warp] = sum;
                part[parity][1][warp] = peak;
            }
            __syncthreads();  // the other parity's slots are free: every thread has read them before this barrier
            sum = lane < nwarps ? part[parity][0][lane] : 0.0f;
            peak = lane < nwarps ? part[parity][1][lane] : 0.0f;
            parity ^= 1;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                if (kNorm) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                peak = max_nan(peak, __shfl_xor_sync(0xffffffffu, peak, o));
            }
        }
        const float r = kNorm ? 1.0f / sqrtf(sum / (float)a.H + a.eps) : 1.0f;
        if (kNorm) peak *= r;
        const bool zero = peak < kZeroRow;  // false for NaN
        const float inv = zero ? 0.0f : kLow8 / peak;
        if (q && tid == 0)
            st_v4(q + a.H, make_uint4(__float_as_uint(zero ? 0.0f : peak / kLow8), 0, 0, 0));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = tid + j * width;
            if (i >= nvec) break;
            if (kNorm) {
#pragma unroll
                for (int p = 0; p < 8; ++p) t[j][p] *= r;
                if (a.y)
                    st_v4(a.y + at + (size_t)i * 8, make_uint4(bf16x2(t[j][0], t[j][1]), bf16x2(t[j][2], t[j][3]),
                                                               bf16x2(t[j][4], t[j][5]), bf16x2(t[j][6], t[j][7])));
            }
            if (q) {
                uint2 v;
                v.x = e4m3x2(t[j][0] * inv, t[j][1] * inv) | e4m3x2(t[j][2] * inv, t[j][3] * inv) << 16;
                v.y = e4m3x2(t[j][4] * inv, t[j][5] * inv) | e4m3x2(t[j][6] * inv, t[j][7] * inv) << 16;
                *reinterpret_cast<uint2 *>(q + (size_t)i * 8) = v;
            }
        }
    }
}

template <int V, int kThreads, int kBlocks, bool kNorm, bool kWarp = false>
cudaError_t launch_rows(const a2av_plan_s &p, const NormArgs &a, cudaStream_t s) {
    const int block = kWarp ? kThreads : ((a.H / 8 + V - 1) / V + 31) / 32 * 32;
    const long long cap = (long long)p.num_sms * (kThreads * kBlocks / block);
    const long long want = kWarp ? (a.rows + (long long)block / 32 - 1) / (block / 32) : a.rows;
    return launch_pdl(norm_kernel<V, kThreads, kBlocks, kNorm, kWarp>, (int)(want < cap ? want : cap), block, 0, s, a);
}

}  // namespace

// Two vectors per thread and room for 64 registers (two blocks of 512 threads
// per SM): with the next row's loads held in registers that is 64 KiB in
// flight per SM.  65,536 x 7168 to 8 bits: 492 us (6.68 TB/s); one vector and
// 1024 threads 586 us, two and three blocks (42 registers, spills) 621 us,
// four vectors 611-676 us.  Without the norm the row needs fewer registers and
// a third block pays: 32,768 x 2048 33.3 us against 37.1 us.  Longer rows take
// as many threads as a block has.  Rows of up to 256, one vector a lane, take a warp each,
// without the block's barrier: 65,536 x 256 to 8 bits 22.6 us against 30.3, without the norm 12.7 against 17.8;
// at 512 two vectors a lane lose (46.4 us against 43.9).
cudaError_t launch_norm(const a2av_plan_s &p, const NormArgs &a, bool norm, cudaStream_t s) {
    if (a.H <= 256)
        return norm ? launch_rows<1, 256, 5, true, true>(p, a, s) : launch_rows<1, 256, 5, false, true>(p, a, s);
    if (a.H > 16384) return norm ? launch_rows<4, 1024, 1, true>(p, a, s) : launch_rows<4, 1024, 1, false>(p, a, s);
    if (a.H > 8192) return norm ? launch_rows<2, 1024, 1, true>(p, a, s) : launch_rows<2, 1024, 1, false>(p, a, s);
    return norm ? launch_rows<2, 512, 2, true>(p, a, s) : launch_rows<2, 512, 3, false>(p, a, s);
}

}  // namespace a2av
