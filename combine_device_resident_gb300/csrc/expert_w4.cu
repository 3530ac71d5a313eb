// The experts' products with 4-bit weights and group scales, for few rows:
//
//   y[r][n] = act( sum_g s[n][g] * sum_{k in g} (q[n][k] - 8) * x[r][k] )
//
// Bound by the weights' bytes (half a byte each), so everything is arranged
// around streaming them: a block of eight warps takes 16 or 32 weight rows,
// the warps share out K in spans of 256, and each warp keeps its own ring of
// TMA boxes (32 rows x 128 bytes) in flight, across work items too.  A word of
// eight 4-bit weights gives four bf16 pairs by a mask and an or each (q | 0x4300
// is 128 + q) and an exact subtraction; the pairs are A fragments of the 16x8x16
// matrix instruction, whose legacy form is the right one here: the product
// needs 2*rows flops per weight, far below any tensor limit, and its operands
// come out of registers.  Each group's sum is scaled in fp32, so no weight is
// rounded.  The warps' partial sums meet in shared memory in a fixed order.
#include <cuda_bf16.h>

#include "expert_common.cuh"

namespace a2av {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kSpan = 256;     // K of a TMA box: 128 bytes of a weight row
constexpr int kStages = 4;     // boxes of 16 weight rows in flight per warp (half as many of 32)
constexpr int kMaxRows = 32;   // expert rows per work item

struct Shared4 {
    uint64_t full[kWarps][kStages];
    uint32_t abort;
    int32_t warp_sum[kWarps];
};

// Bits i*4 and 16+i*4 of a word: k = 2i and 2i+1 as bf16, minus 8.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(v) : "r"(w >> (4 * i)));  // (w & mask) | 128.0
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), __nv_bfloat162{__float2bfloat16(136.0f), __float2bfloat16(136.0f)});
    return *reinterpret_cast<const uint32_t *>(&d);
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }

struct Item {
    int e, row, rows, block;
};

__device__ __forceinline__ Item item_at(long long t, const int32_t *start, const int32_t *count, const int32_t *pre,
                                        int E, int blocks) {
    Item w;
    w.e = expert_of(t, pre, E, blocks);
    const int in = (int)(t - (long long)pre[w.e] * blocks);
    const int chunks = (count[w.e] + kMaxRows - 1) / kMaxRows;  // the chunks of one weight block follow each other
    w.block = in / chunks;
    const int first = in % chunks * kMaxRows;
    w.row = start[w.e] + first;
    w.rows = min(kMaxRows, count[w.e] - first);
    return w;
}

// One box: kRows weight rows x kSpan of K for kNT*8 expert rows, into acc.
// Weight rows of tile m: `lower(m) + g` and `upper(m) + g`, g = lane / 4.
template <int kMT, int kNT, bool kSwiglu>
__device__ __forceinline__ void accumulate(const uint32_t *box, const MatmulArgs &a, const Item &w, int k0,
                                           float (&acc)[kMT][4][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int words = min(kSpan, a.K - k0) / 32;  // 32-wide steps; K is a multiple of 32
    const int groups = a.K / a.group, per = a.group / 32;
    const uint16_t *x = reinterpret_cast<const uint16_t *>(a.x) + (size_t)w.row * a.K + k0 + t * 8;
    const uint16_t *scale[kMT][2];
    int low[kMT][2];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // swiglu: the lower rows are gates, the upper ones the same channels' ups
            low[m][h] = kSwiglu ? h * 8 * kMT + m * 8 : m * 16 + h * 8;
            const int chan = w.block * (kSwiglu ? 8 : 16) * kMT + (kSwiglu ? m * 8 : m * 16 + h * 8) + g;
            const size_t row = (size_t)w.e * a.N * (kSwiglu ? 2 : 1) + (kSwiglu && h ? a.N : 0) + min(chan, a.N - 1);
            scale[m][h] = static_cast<const uint16_t *>(a.w_scale) + row * groups;
        }
    for (int j0 = 0; j0 < words; j0 += per) {  // one group of K at a time
        float part[kMT][kNT][4] = {};
        float s[kMT][2];
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) s[m][h] = bf16_at(scale[m][h] + (k0 + j0 * 32) / a.group);
#pragma unroll 4
        for (int j = j0; j < j0 + per; ++j) {
            uint4 b[kNT];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
                b[n] = n * 8 + g < w.rows ? __ldg(reinterpret_cast<const uint4 *>(x + (size_t)(n * 8 + g) * a.K + j * 32))
                                          : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                const uint32_t w0 = box[(low[m][0] + g) * 32 + ((j ^ g) * 4 + t)];
                const uint32_t w1 = box[(low[m][1] + g) * 32 + ((j ^ g) * 4 + t)];
                const uint32_t p0 = pair_of(w0, 0), p1 = pair_of(w0, 1), p2 = pair_of(w0, 2), p3 = pair_of(w0, 3);
                const uint32_t q0 = pair_of(w1, 0), q1 = pair_of(w1, 1), q2 = pair_of(w1, 2), q3 = pair_of(w1, 3);
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    mma16816(part[m][n], p0, q0, p1, q1, b[n].x, b[n].y);
                    mma16816(part[m][n], p2, q2, p3, q3, b[n].z, b[n].w);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                acc[m][n][0] = fmaf(s[m][0], part[m][n][0], acc[m][n][0]);
                acc[m][n][1] = fmaf(s[m][0], part[m][n][1], acc[m][n][1]);
                acc[m][n][2] = fmaf(s[m][1], part[m][n][2], acc[m][n][2]);
                acc[m][n][3] = fmaf(s[m][1], part[m][n][3], acc[m][n][3]);
            }
    }
}

// kMT: 16-row weight tiles per work item.
template <int kMT, bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 2) expert_w4_kernel(const __grid_constant__ CUtensorMap map_w,
                                                                const MatmulArgs a) {
    constexpr int kRows = kMT * 16, kBoxBytes = kRows * 128, kRing = kStages / kMT;
    constexpr int kChan = kSwiglu ? kRows / 2 : kRows;  // output channels per work item
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    float *parts = reinterpret_cast<float *>(ring + kWarps * kRing * kBoxBytes);  // [warp][kRows][kMaxRows + 1]
    Shared4 *sh = reinterpret_cast<Shared4 *>(parts + kWarps * kRows * (kMaxRows + 1));
    const int E = a.g.E;
    int32_t *start = reinterpret_cast<int32_t *>(sh + 1);
    int32_t *count = start + E;
    int32_t *pre = count + E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < kWarps * kRing) mbar_init(&sh->full[tid / kRing][tid % kRing], 1);
    if (tid == 0) {
        sh->abort = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w));
    }
    fence_mbar_init();
    grid_dependency_wait();
    const int total = place_experts<kThreads>(a, kMaxRows, start, count, pre, sh->warp_sum);  // ends in a barrier
    const int blocks = (a.N + kChan - 1) / kChan;
    const long long items = (long long)total * blocks;
    const int spans = (a.K + kSpan - 1) / kSpan;

    uint8_t *mine = ring + warp * kRing * kBoxBytes;
    // The warp's boxes in order: of item i of this block, spans (warp + i) % kWarps, + kWarps, ...; the
    // rotation evens out a K whose spans do not divide by the warps.
    long long put_t = blockIdx.x;
    int put_i = 0, put_span = warp;
    uint32_t put = 0, got = 0;  // boxes issued and consumed
    bool ok = true;
    auto issue = [&] {  // the next box of this warp, if there is one
        while (put_t < items && put_span >= spans) {
            put_t += gridDim.x;
            ++put_i;
            put_span = (warp + put_i) % kWarps;
        }
        if (put_t >= items) return;
        if (lane == 0) {
            const Item w = item_at(put_t, start, count, pre, E, blocks);
            uint64_t *bar = &sh->full[warp][put % kRing];
            mbar_arrive_expect_tx(bar, kBoxBytes);
            asm volatile(
                "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
                "%5}], [%6];" ::"r"(smem_u32(mine + put % kRing * kBoxBytes)),
                "l"(&map_w), "r"(put_span * (kSpan / 8)), "r"(w.block * kChan), "r"(0), "r"(w.e), "r"(smem_u32(bar))
                : "memory");
        }
        put_span += kWarps;
        ++put;
    };
    for (int i = 0; i < kRing; ++i) issue();

    int i = 0;
    for (long long t = blockIdx.x; t < items; t += gridDim.x, ++i) {
        const Item w = item_at(t, start, count, pre, E, blocks);
        float acc[kMT][4][4] = {};
        for (int span = (warp + i) % kWarps; ok && span < spans; span += kWarps) {
            const int s = got % kRing;
            const bool in = mbar_wait_bounded(&sh->full[warp][s], (got / kRing) & 1, a.wait_polls);
            if (!all_of(in)) {
                ok = false;
                break;
            }
            const uint32_t *box = reinterpret_cast<const uint32_t *>(mine + s * kBoxBytes);
            if (w.rows <= 8) accumulate<kMT, 1, kSwiglu>(box, a, w, span * kSpan, acc);
            else if (w.rows <= 16) accumulate<kMT, 2, kSwiglu>(box, a, w, span * kSpan, acc);
            else accumulate<kMT, 4, kSwiglu>(box, a, w, span * kSpan, acc);
            ++got;
            __syncwarp();  // every lane has read the box
            issue();
        }
        if (!ok && lane == 0) {
            sh->abort = 1;
            atomicOr(a.status, kDevWaitTimeout);
        }
        const int g = lane >> 2, q = lane & 3;
        float *p = parts + warp * kRows * (kMaxRows + 1);
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n * 8 < w.rows) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        p[(m * 16 + (c >> 1) * 8 + g) * (kMaxRows + 1) + n * 8 + q * 2 + (c & 1)] = acc[m][n][c];
                }
        __syncthreads();
        if (*(volatile uint32_t *)&sh->abort == 0)
            for (int o = tid; o < kChan * w.rows; o += kThreads) {
                const int chan = o % kChan, r = o / kChan;
                const int lower = kSwiglu ? chan / 8 * 16 + chan % 8 : chan;
                float sum = 0.0f, up = 0.0f;
#pragma unroll
                for (int v = 0; v < kWarps; ++v) {
                    sum += parts[(v * kRows + lower) * (kMaxRows + 1) + r];
                    if (kSwiglu) up += parts[(v * kRows + lower + 8) * (kMaxRows + 1) + r];
                }
                const float out = kSwiglu ? __fdividef(sum, 1.0f + __expf(-sum)) * up : sum;
                const int n = w.block * kChan + chan;
                if (n < a.N) a.y[(size_t)(w.row + r) * a.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(out));
            }
        __syncthreads();
    }
    if (!ok)  // given up: the boxes that were issued land before the block ends
        for (; got < put; ++got) mbar_wait_bounded(&sh->full[warp][got % kRing], (got / kRing) & 1);
}

// ---- many work items: rows shared out among the warps -------------------------
//
// A producer warp fills a ring of stages with the weights' boxes (every
// consumer warp's kMT*16 rows at once) and the expert rows' same span of K; x is then read
// once per block instead of once per warp, and a consumer keeps whole sums.
constexpr int kXPitch = kSpan * 2 + 64;  // a row of x in a stage; 64 more bytes spread two rows over all banks

template <int kW, int kMT, int kNT, bool kSwiglu, int kPer>
__device__ __forceinline__ void stage_sums(const uint8_t *weights, const uint8_t *x, int words, const float *scale,
                                           float (&acc)[kMT][4][4]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    constexpr int kChan = kW * kMT * (kSwiglu ? 8 : 16);
#pragma unroll
    for (int j0 = 0; j0 < 8; j0 += kPer) {
        if (j0 >= words) break;
        float part[kMT][kNT][4] = {};
#pragma unroll
        for (int j = j0; j < j0 + kPer; ++j) {
            uint4 b[kNT];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
                b[n] = *reinterpret_cast<const uint4 *>(x + (n * 8 + g) * kXPitch + j * 64 + t * 16);
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
                const int low = kSwiglu ? (warp * kMT + m) * 8 : (warp * kMT + m) * 16;
                const int high = kSwiglu ? kChan + low : low + 8;
                const uint32_t at = (j ^ g) * 16 + t * 4 + g * 128;
                const uint32_t w0 = *reinterpret_cast<const uint32_t *>(weights + low * 128 + at);
                const uint32_t w1 = *reinterpret_cast<const uint32_t *>(weights + high * 128 + at);
                const uint32_t p0 = pair_of(w0, 0), p1 = pair_of(w0, 1), p2 = pair_of(w0, 2), p3 = pair_of(w0, 3);
                const uint32_t q0 = pair_of(w1, 0), q1 = pair_of(w1, 1), q2 = pair_of(w1, 2), q3 = pair_of(w1, 3);
#pragma unroll
                for (int n = 0; n < kNT; ++n) {
                    mma16816(part[m][n], p0, q0, p1, q1, b[n].x, b[n].y);
                    mma16816(part[m][n], p2, q2, p3, q3, b[n].z, b[n].w);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            const float s0 = scale[(j0 / kPer * kMT + m) * 2], s1 = scale[(j0 / kPer * kMT + m) * 2 + 1];
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                acc[m][n][0] = fmaf(s0, part[m][n][0], acc[m][n][0]);
                acc[m][n][1] = fmaf(s0, part[m][n][1], acc[m][n][1]);
                acc[m][n][2] = fmaf(s1, part[m][n][2], acc[m][n][2]);
                acc[m][n][3] = fmaf(s1, part[m][n][3], acc[m][n][3]);
            }
        }
    }
}

struct SharedRows {
    uint64_t full[4], empty[4];
    uint32_t abort;
    int32_t warp_sum[32];
};

// kPer: 32-wide steps per group of K.
template <int kW, int kMT, bool kSwiglu, int kPer, int kRing>
__global__ void __launch_bounds__((kW + 1) * 32, 2)
    expert_w4_rows_kernel(const __grid_constant__ CUtensorMap map_w, const MatmulArgs a) {
    constexpr int kRows = kW * kMT * 16, kChan = kSwiglu ? kRows / 2 : kRows, kBlock = (kW + 1) * 32;
    constexpr int kWBytes = kRows * 128, kStage = kWBytes + (kMaxRows * kXPitch + 1023) / 1024 * 1024;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    SharedRows *sh = reinterpret_cast<SharedRows *>(ring + kRing * kStage);
    const int E = a.g.E;
    int32_t *start = reinterpret_cast<int32_t *>(sh + 1);
    int32_t *count = start + E;
    int32_t *pre = count + E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], kW);
        }
        sh->abort = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w));
    }
    grid_dependency_wait();
    const int total = place_experts<kBlock>(a, kMaxRows, start, count, pre, sh->warp_sum);  // ends in a barrier
    const int blocks = (a.N + kChan - 1) / kChan;
    const long long items = (long long)total * blocks;
    const int spans = (a.K + kSpan - 1) / kSpan;

    if (warp == kW) {
        int s = 0;
        uint32_t round = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < items; t += gridDim.x) {
            const Item w = item_at(t, start, count, pre, E, blocks);
            const uint8_t *x = a.x + (size_t)(w.row + lane) * a.x_pitch;
            for (int span = 0; span < spans; ++span) {
                if (round > 0) {
                    const bool in = wait_or_abort(&sh->empty[s], (round - 1) & 1, a.wait_polls, &sh->abort, a.status);
                    if (!all_of(in)) {
                        ok = false;
                        break;
                    }
                }
                uint8_t *stage = ring + s * kStage;
                const uint32_t bytes = min(kSpan, a.K - span * kSpan) * 2;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh->full[s], kWBytes + w.rows * bytes);
                    asm volatile(
                        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                        "%3, %4, %5}], [%6];" ::"r"(smem_u32(stage)),
                        "l"(&map_w), "r"(span * (kSpan / 8)), "r"(w.block * kChan), "r"(0), "r"(w.e),
                        "r"(smem_u32(&sh->full[s]))
                        : "memory");
                }
                __syncwarp();
                if (lane < w.rows)
                    bulk_load(stage + kWBytes + lane * kXPitch, x + (size_t)span * kSpan * 2, bytes, &sh->full[s]);
                if (++s == kRing) {
                    s = 0;
                    ++round;
                }
            }
        }
        if (lane == 0)  // every load that was issued lands before the block ends, also if the others gave up
            for (int i = 0; i < kRing; ++i) {
                const uint32_t fills = round + (i < s ? 1 : 0);
                if (fills > 0) mbar_wait_bounded(&sh->full[i], (fills - 1) & 1);
            }
    } else {
        constexpr int kGroups = 8 / kPer;  // groups of a stage
        const int g = lane >> 2, q = lane & 3;
        const int groups = a.K / a.group;
        int s = 0;
        uint32_t round = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < items; t += gridDim.x) {
            const Item w = item_at(t, start, count, pre, E, blocks);
            const uint16_t *from[kMT][2];
#pragma unroll
            for (int m = 0; m < kMT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int chan = w.block * kChan + (kSwiglu ? (warp * kMT + m) * 8 : (warp * kMT + m) * 16 + h * 8) + g;
                    const size_t row = (size_t)w.e * a.N * (kSwiglu ? 2 : 1) + (kSwiglu && h ? a.N : 0) + min(chan, a.N - 1);
                    from[m][h] = static_cast<const uint16_t *>(a.w_scale) + row * groups;
                }
            // the scales of a stage, one stage ahead
            uint16_t next[kGroups * kMT * 2];
            auto fetch = [&](int span) {
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
#pragma unroll
                    for (int m = 0; m < kMT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = min(span * kGroups + i, groups - 1);
                            next[(i * kMT + m) * 2 + h] = __ldg(from[m][h] + at);
                        }
            };
            fetch(0);
            float acc[kMT][4][4] = {};
            for (int span = 0; span < spans; ++span) {
                float scale[kGroups * kMT * 2];
#pragma unroll
                for (int i = 0; i < kGroups * kMT * 2; ++i) scale[i] = __uint_as_float((uint32_t)next[i] << 16);
                fetch(min(span + 1, spans - 1));
                const bool in = wait_or_abort(&sh->full[s], round & 1, a.wait_polls, &sh->abort, a.status);
                if (!all_of(in)) {
                    ok = false;
                    break;
                }
                const uint8_t *stage = ring + s * kStage;
                const int words = min(kSpan, a.K - span * kSpan) / 32;
                if (w.rows <= 8) stage_sums<kW, kMT, 1, kSwiglu, kPer>(stage, stage + kWBytes, words, scale, acc);
                else if (w.rows <= 16) stage_sums<kW, kMT, 2, kSwiglu, kPer>(stage, stage + kWBytes, words, scale, acc);
                else stage_sums<kW, kMT, 4, kSwiglu, kPer>(stage, stage + kWBytes, words, scale, acc);
                __syncwarp();  // every lane has read the stage
                if (lane == 0) mbar_arrive(&sh->empty[s]);
                if (++s == kRing) {
                    s = 0;
                    ++round;
                }
            }
            if (!ok) break;
#pragma unroll
            for (int m = 0; m < kMT; ++m)
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = n * 8 + q * 2 + c;
                        const int chan = w.block * kChan + (warp * kMT + m) * (kSwiglu ? 8 : 16) + g;
                        if (r >= w.rows) continue;
                        uint16_t *y = a.y + (size_t)(w.row + r) * a.N + chan;
                        const float lo = acc[m][n][c], hi = acc[m][n][c + 2];
                        if (kSwiglu) {
                            if (chan < a.N)
                                y[0] = __bfloat16_as_ushort(
                                    __float2bfloat16_rn(__fdividef(lo, 1.0f + __expf(-lo)) * hi));
                        } else {
                            if (chan < a.N) y[0] = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
                            if (chan + 8 < a.N) y[8] = __bfloat16_as_ushort(__float2bfloat16_rn(hi));
                        }
                    }
        }
    }
}

cudaError_t map_words(CUtensorMap *m, const MatmulArgs &a, bool swiglu, int chan) {
    const cuuint64_t halves = swiglu ? 2 : 1, row = (cuuint64_t)a.K / 2;
    // w as [E][gate, up][N][K/8]
    const cuuint64_t dims[4] = {(cuuint64_t)a.K / 8, (cuuint64_t)a.N, halves, (cuuint64_t)a.g.E};
    const cuuint64_t strides[3] = {row, a.N * row, halves * a.N * row};
    const cuuint32_t box[4] = {kSpan / 8, (cuuint32_t)chan, (cuuint32_t)halves, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, a.w, dims, strides, box) ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kW, int kMT, bool kSwiglu, int kPer, int kRing>
cudaError_t launch_w4_rows(const a2av_plan_s &p, const MatmulArgs &a, cudaStream_t s) {
    constexpr int kRows = kW * kMT * 16, kChan = kSwiglu ? kRows / 2 : kRows;
    constexpr int kStage = kRows * 128 + (kMaxRows * kXPitch + 1023) / 1024 * 1024;
    CUtensorMap m;
    cudaError_t e = map_words(&m, a, kSwiglu, kChan);
    if (e != cudaSuccess) return e;
    const auto kernel = expert_w4_rows_kernel<kW, kMT, kSwiglu, kPer, kRing>;
    const size_t smem = 1024 + (size_t)kRing * kStage + sizeof(SharedRows) + (size_t)a.g.E * 3 * 4;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.g.R * a.g.T * a.g.k;
    const long long most = ((rows < a.g.E ? rows : a.g.E) + rows / kMaxRows) * ((a.N + kChan - 1) / kChan);
    const int grid = (int)(most < 2 * p.num_sms ? most : 2 * p.num_sms);
    return launch_pdl(kernel, grid, (kW + 1) * 32, smem, s, m, a);
}

template <int kW, int kMT, bool kSwiglu, int kRing>
cudaError_t launch_w4_group(const a2av_plan_s &p, const MatmulArgs &a, cudaStream_t s) {
    return a.group == 32   ? launch_w4_rows<kW, kMT, kSwiglu, 1, kRing>(p, a, s)
           : a.group == 64 ? launch_w4_rows<kW, kMT, kSwiglu, 2, kRing>(p, a, s)
                           : launch_w4_rows<kW, kMT, kSwiglu, 4, kRing>(p, a, s);
}

template <int kMT, bool kSwiglu>
cudaError_t launch_w4(const a2av_plan_s &p, const MatmulArgs &a, cudaStream_t s) {
    constexpr int kRows = kMT * 16, kChan = kSwiglu ? kRows / 2 : kRows;
    CUtensorMap m;
    cudaError_t e = map_words(&m, a, kSwiglu, kChan);
    if (e != cudaSuccess) return e;
    const size_t smem = 1024 + (size_t)kWarps * (kStages / kMT) * kRows * 128 + (size_t)kWarps * kRows * (kMaxRows + 1) * 4 +
                        sizeof(Shared4) + (size_t)a.g.E * 3 * 4;
    e = cudaFuncSetAttribute(expert_w4_kernel<kMT, kSwiglu>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.g.R * a.g.T * a.g.k;
    const long long most = ((rows < a.g.E ? rows : a.g.E) + rows / kMaxRows) * ((a.N + kChan - 1) / kChan);
    const int grid = (int)(most < 2 * p.num_sms ? most : 2 * p.num_sms);
    return launch_pdl(expert_w4_kernel<kMT, kSwiglu>, grid, kThreads, smem, s, m, a);
}

}  // namespace

cudaError_t launch_expert_w4(const a2av_plan_s &p, const MatmulArgs &a, bool swiglu, cudaStream_t s) {
    const long long rows = (long long)a.g.R * a.g.T * a.g.k, experts = rows < a.g.E ? rows : a.g.E;
    const bool wide = experts * (swiglu ? 2 : 1) * a.N / 128 >= 2 * p.num_sms;
    if (wide) return swiglu ? launch_w4_group<8, 1, true, 3>(p, a, s) : launch_w4_group<8, 1, false, 3>(p, a, s);
    return swiglu ? launch_w4<1, true>(p, a, s) : launch_w4<1, false>(p, a, s);
}

}  // namespace a2av
