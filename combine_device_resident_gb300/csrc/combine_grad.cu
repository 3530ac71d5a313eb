// The combine's gradient: for every assignment (t, j) with slot s,
//
//   d_y[s] = bf16(gate * d_out[t]),   d_gate = <y[s], d_out[t]>   (fp32 sums of exact products)
//
// One block per token: its row of d_out stays in registers while the k rows of y come in and the k rows of d_y go out,
// so everything moves once.  Bound by HBM.  Rows of up to 16,384 (piped): while an assignment is worked on, the next one's
// row of y is on its way, with the next token's row of d_out after the last, and the slot after that; the blocks' loads
// then overlap their stores and sums.  Longer rows go in pieces, without.
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

template <int V, bool kRows, bool kGates>
__global__ void __launch_bounds__(kMaxThreads, 4 / V) combine_grad_piped_kernel(const CombineGradArgs a) {
    __shared__ float part[2][kMaxTopk][kMaxThreads / 32];  // [token parity]
    const int k = a.g.k, H = a.g.H, nvec = H / 8, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nwarps = blockDim.x >> 5;
    const long long ntok = (long long)a.g.R * a.g.T;
    auto active = [&](long long u) {  // from u on, in the block's steps
        if (a.num_tokens)
            for (; u < ntok; u += gridDim.x) {
                const int s = (int)(u / a.g.T);
                if (u - (long long)s * a.g.T < active_tokens(a.num_tokens, s, a.g.T)) break;
            }
        return u;
    };
    struct Item {  // an assignment
        long long u;
        int j;
        int32_t slot;  // negative: none
        float gate;
    };
    auto ask = [&](Item &i) {
        i.slot = -1;
        i.gate = 0.0f;
        if (i.u >= ntok) return;
        i.slot = __ldg(a.slot_map + i.u * k + i.j);
        if (kRows) i.gate = __ldg(a.gate + i.u * k + i.j);
    };
    auto after = [&](const Item &i) {
        Item n = i;
        if (++n.j == k) {
            n.j = 0;
            n.u = i.u < ntok ? active(i.u + gridDim.x) : i.u;
        }
        ask(n);
        return n;
    };
    auto load = [&](const uint16_t *row, uint4 (&to)[V]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = tid + v * blockDim.x;
            if (i < nvec) to[v] = ld_row(row + (size_t)i * 8);
        }
    };
    auto fits = [&](const Item &i) { return i.slot >= 0 && i.slot < a.arena_rows; };
    grid_dependency_wait();
    Item now;
    now.u = active(blockIdx.x);
    now.j = 0;
    ask(now);
    Item next = after(now);
    uint4 d[V], y[V], dn[V], yn[V];
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = y[v] = dn[v] = yn[v] = make_uint4(0, 0, 0, 0);  // behind the row's end for good
    if (now.u < ntok) {
        load(a.d_out + (size_t)now.u * H, d);
        if (kGates && fits(now)) load(a.y + (size_t)now.slot * H, y);
    }
    int parity = 0;
    while (now.u < ntok) {
        const bool last = now.j == k - 1;
        if (kGates && fits(next)) load(a.y + (size_t)next.slot * H, yn);
        if (last && next.u < ntok) load(a.d_out + (size_t)next.u * H, dn);
        const Item then = after(next);
        if (now.slot >= a.arena_rows && tid == 0) atomicOr(a.status, kDevBadSlot);
        if (kRows && fits(now)) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = tid + v * blockDim.x;
                if (i < nvec) st_v4(a.d_y + (size_t)now.slot * H + (size_t)i * 8, scaled8(d[v], now.gate));
            }
        }
        if (kGates) {
            float dot = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) dot = dot8(d[v], y[v], dot);
            dot = warp_sum(fits(now) ? dot : 0.0f);
            if (lane == 0) part[parity][now.j][warp] = dot;
            if (last) {
                __syncthreads();  // the other parity's sums are written out by now, before this barrier
                if (tid < k) {
                    float sum = 0.0f;
                    for (int w = 0; w < nwarps; ++w) sum += part[parity][tid][w];
                    a.d_gate[now.u * k + tid] = sum;
                }
                parity ^= 1;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            y[v] = yn[v];
            if (last) d[v] = dn[v];
        }
        now = next;
        next = then;
    }
}

// Two vectors a thread where the row fits (64 registers, two blocks of 448 per SM for H = 7168): 65,536 x 7168, top-8:
// 2464 us (6.48 TB/s); four vectors and 224 threads 2708-2892 us at 64 to 117 registers, the same without the loads
// ahead 2671 us; 2,040 x 5120, top-1: 10.8 us against 12.8-16.5 and 13.9.
template <int V, bool kRows, bool kGates>
cudaError_t launch_piped(const a2av_plan_s &p, const CombineGradArgs &a, cudaStream_t s) {
    const int block = ((a.g.H / 8 + V - 1) / V + 31) / 32 * 32, fit = 65536 / (32 * V) / block;
    const long long ntok = (long long)a.g.R * a.g.T, cap = (long long)p.num_sms * (fit < 1 ? 1 : fit > 32 ? 32 : fit);
    return launch_pdl(combine_grad_piped_kernel<V, kRows, kGates>, (int)(ntok < cap ? ntok : cap), block, 0, s, a);
}

template <int V>
cudaError_t launch_piped_form(const a2av_plan_s &p, const CombineGradArgs &a, cudaStream_t s) {
    if (!a.d_y) return launch_piped<V, false, true>(p, a, s);
    return a.d_gate ? launch_piped<V, true, true>(p, a, s) : launch_piped<V, true, false>(p, a, s);
}

}  // namespace

cudaError_t launch_combine_grad(const a2av_plan_s &p, const CombineGradArgs &a, cudaStream_t s) {
    const int nvec = a.g.H / 8;
    if (nvec <= 2 * kMaxThreads) return launch_piped_form<2>(p, a, s);
    if (nvec <= 4 * kMaxThreads) return launch_piped_form<4>(p, a, s);
    const long long ntok = (long long)a.g.R * a.g.T, cap = (long long)p.num_sms * 2;
    return launch_pdl(combine_grad_kernel, (int)(ntok < cap ? ntok : cap), kMaxThreads, 0, s, a);
}

}  // namespace a2av
