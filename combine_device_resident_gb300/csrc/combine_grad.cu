// The combine's gradient: for every assignment (t, j) with slot s,
//
//   d_y[s] = bf16(gate * d_out[t]),   d_gate = <y[s], d_out[t]>   (fp32 sums of exact products)
//
// One block per token: its row of d_out stays in registers while the k rows of y come in and the k rows of d_y go out,
// so everything moves once.  Bound by HBM.
#include "block_ops.cuh"
#include "row_math.cuh"

namespace a2av {
namespace {

constexpr int kVec = 4;  // 16-byte vectors of a row per thread at a time
constexpr int kMaxThreads = 512;

__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float s) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(hi_f(x[i]), hi_f(y[i]), fmaf(lo_f(x[i]), lo_f(y[i]), s));
    return s;
}
__device__ __forceinline__ uint4 scaled8(const uint4 &a, float w) {
    return make_uint4(bf16x2(lo_f(a.x) * w, hi_f(a.x) * w), bf16x2(lo_f(a.y) * w, hi_f(a.y) * w),
                      bf16x2(lo_f(a.z) * w, hi_f(a.z) * w), bf16x2(lo_f(a.w) * w, hi_f(a.w) * w));
}

__global__ void __launch_bounds__(kMaxThreads) combine_grad_kernel(const CombineGradArgs a) {
    __shared__ int32_t slots[kMaxTopk];
    __shared__ float gates[kMaxTopk], part[kMaxTopk][kMaxThreads / 32];
    const int k = a.g.k, H = a.g.H, nvec = H / 8, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nwarps = blockDim.x >> 5, ntok = a.g.R * a.g.T;
    grid_dependency_wait();
    for (long long u = blockIdx.x; u < ntok; u += gridDim.x) {
        if (a.num_tokens) {
            const int s = (int)(u / a.g.T);
            if (u - (long long)s * a.g.T >= active_tokens(a.num_tokens, s, a.g.T)) continue;
        }
        if (tid < k) {
            int32_t s = __ldg(a.slot_map + u * k + tid);
            if (s >= a.arena_rows) {
                atomicOr(a.status, kDevBadSlot);
                s = -1;
            }
            slots[tid] = s;
            gates[tid] = a.d_y ? __ldg(a.gate + u * k + tid) : 0.0f;
        }
        __syncthreads();
        for (int c = tid; c - tid < nvec; c += blockDim.x * kVec) {  // the whole block goes on to the next piece
            uint4 d[kVec];
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const int i = c + v * blockDim.x;
                d[v] = i < nvec ? ld_row(a.d_out + (size_t)u * H + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
            }
            for (int j = 0; j < k; ++j) {
                const int32_t s = slots[j];
                float dot = 0.0f;
                if (s >= 0) {
                    const size_t at = (size_t)s * H;
                    if (a.d_gate) {
                        uint4 y[kVec];
#pragma unroll
                        for (int v = 0; v < kVec; ++v) {
                            const int i = c + v * blockDim.x;
                            y[v] = i < nvec ? ld_row(a.y + at + (size_t)i * 8) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int v = 0; v < kVec; ++v) dot = dot8(d[v], y[v], dot);
                    }
                    if (a.d_y) {
                        const float w = gates[j];
#pragma unroll
                        for (int v = 0; v < kVec; ++v) {
                            const int i = c + v * blockDim.x;
                            if (i < nvec) st_v4(a.d_y + at + (size_t)i * 8, scaled8(d[v], w));
                        }
                    }
                }
                if (a.d_gate) {
                    dot = warp_sum(dot);
                    if (lane == 0) part[j][warp] = (c < (int)(blockDim.x * kVec) ? 0.0f : part[j][warp]) + dot;
                }
            }
        }
        __syncthreads();
        if (a.d_gate && tid < k) {
            float dot = 0.0f;
            for (int w = 0; w < nwarps; ++w) dot += part[tid][w];
            a.d_gate[u * k + tid] = dot;
        }
    }
}

}  // namespace

cudaError_t launch_combine_grad(const a2av_plan_s &p, const CombineGradArgs &a, cudaStream_t s) {
    const int nvec = a.g.H / 8;
    const int want = ((nvec + kVec - 1) / kVec + 31) / 32 * 32, block = want < kMaxThreads ? want : kMaxThreads;
    const long long ntok = (long long)a.g.R * a.g.T, per_sm = 1024 / block < 16 ? 1024 / block : 16;
    const long long cap = (long long)p.num_sms * per_sm;
    return launch_pdl(combine_grad_kernel, (int)(ntok < cap ? ntok : cap), block, 0, s, a);
}

}  // namespace a2av
