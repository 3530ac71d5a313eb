// What the experts' products share: where each expert's rows lie, the order of
// the work, tensor maps, and a wait that ends when another warp gave up.
#pragma once

#include <cuda.h>

#include <atomic>

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

// g / (1 + exp(-g)) * u.  The power is exp(-|g|), at most 1, so that the divisor lies between 1 and 2: with exp(-g) it
// grows past 2^126 at gates below -87.3, where the fast division gives 0.  Both are the fast forms, some
// (5 + 1.2 |g|) * 2^-23 off, far below the bf16 the result is rounded to.
__device__ __forceinline__ float swiglu(float g, float u) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g >= 0.0f ? g : g * e, 1.0f + e) * u;
}

// One answer for the warp.
__device__ __forceinline__ bool all_of(bool v) { return __all_sync(0xffffffffu, v); }

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(v));
    return v != 0;
}

// Shared-memory operand descriptor: K-major, 128-byte swizzle, eight-row
// groups 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// All of tensor memory for this block (a whole warp calls these).
__device__ __forceinline__ void tmem_alloc_all(uint32_t *to) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(to)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_all(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}
// D (+)= A B^T, bf16, A in tensor memory; and an arrival once what was issued so far is done.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void mma_commit_one(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// kCols columns of this warp's 32 lanes into registers, which hold them after tmem_wait_ld; 32 columns out of them.
template <int kCols>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[kCols]) {
    static_assert(kCols == 4 || kCols == 8 || kCols == 16 || kCols == 32, "columns");
    if constexpr (kCols == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(addr));
    else if constexpr (kCols == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "r"(addr));
    else if constexpr (kCols == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
              "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
            : "r"(addr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
              "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
              "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
              "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
              "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
            : "r"(addr));
}
// The loads' registers pass through here, so that no use of them moves ahead of the wait.
template <int kLoads, int kCols>
__device__ __forceinline__ void tmem_wait_ld(float (&v)[kLoads][kCols]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int n = 0; n < kCols; ++n) asm volatile("" : "+f"(v[i][n]));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Lets `kernel` take `most` bytes of shared memory, on its first launch on each device.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, std::atomic<uint64_t> &done, int device, size_t most) {
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// A 128-byte-swizzled tensor map with zeros outside; false where the CUDA driver has no such function or refuses.
bool encode_map(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
                const cuuint64_t *strides, const cuuint32_t *box);

}  // namespace a2av
