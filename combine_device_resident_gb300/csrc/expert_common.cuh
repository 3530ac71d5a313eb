// What the experts' products share: where each expert's rows lie, the order of
// the work, tensor maps, and a wait that ends when another warp gave up.
#pragma once

#include <cuda.h>

#include "a2av_internal.cuh"

namespace a2av {

// Rows of expert e in the arena, from the split arrays the dispatch wrote;
// kept inside the arena and, with fixed windows, inside the window (an
// overflowing window's counts go past its end; those rows were dropped).
__device__ __forceinline__ void expert_rows(const MatmulArgs &a, int e, int &row, int &n) {
    const int epr = a.g.epr, d = e / epr, le = e - d * epr;
    const long long cap = a.g.window_mode == A2AV_WINDOW_FIXED ? a.g.window_rows : a.arena_rows;
    const int32_t *off = a.recv_expert_offsets + (size_t)d * a.g.R * epr;  // source 0's row of window d
    long long lo = epr > 1 ? __ldg(off + le) : 0;
    long long hi = le + 1 < epr ? __ldg(off + le + 1) : __ldg(a.recv_total + d);
    const long long base = __ldg(a.window_base + d);
    lo = base + min(max(lo, 0ll), cap);
    hi = base + min(max(hi, 0ll), cap);
    lo = min(max(lo, 0ll), (long long)a.arena_rows);
    hi = min(max(hi, lo), (long long)a.arena_rows);
    row = (int)lo;
    n = (int)(hi - lo);
}

// Fills start[e], count[e] and pre[e] (row tiles of `rows` rows before expert
// e's) for every expert; returns the row tiles of all.  Called by a whole
// block of kThreads; ends in a block barrier.
template <int kThreads>
__device__ __forceinline__ int place_experts(const MatmulArgs &a, int rows, int32_t *start, int32_t *count,
                                             int32_t *pre, int32_t *warp_sum) {
    const int E = a.g.E, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (E + kThreads - 1) / kThreads;  // thread i takes experts [i*per, (i+1)*per)
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        if (e >= E) break;
        int row, n;
        expert_rows(a, e, row, n);
        start[e] = row;
        count[e] = n;
        pre[e] = mine;
        mine += (n + rows - 1) / rows;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    for (int i = 0; i < per; ++i)
        if (tid * per + i < E) pre[tid * per + i] += before;
    __syncthreads();
    return total;
}

// The expert of work item t, each row tile being `ctiles` items: the last
// expert whose first item is not past t (it has rows, as t is below the total).
__device__ __forceinline__ int expert_of(long long t, const int32_t *pre, int E, int ctiles) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)pre[mid] * ctiles <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Bounded wait that also ends when another warp of the block gave up; a
// warp that gives up tells the other block of its pair, too (`peer`, the
// address of that block's flag, or 0).
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, long long limit, uint32_t *abort_flag,
                                              uint32_t *status, uint32_t peer = 0) {
    volatile uint32_t *abort = abort_flag;
    for (long long it = 0; it < limit; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    if (peer) asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(peer) : "memory");
    atomicOr(status, kDevWaitTimeout);
    return false;
}

// One answer for the warp.
__device__ __forceinline__ bool all_of(bool v) { return __all_sync(0xffffffffu, v); }

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(v));
    return v != 0;
}

// A 128-byte-swizzled tensor map with zeros outside; the reason of a failure in the last error.
bool encode_map(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
                const cuuint64_t *strides, const cuuint32_t *box);

}  // namespace a2av
