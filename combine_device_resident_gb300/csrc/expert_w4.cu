// The experts' products with 4-bit weights and group scales, for few rows:
//
//   y[r][n] = act( sum_g s[n][g] * sum_{k in g} (q[n][k] - 8) * x[r][k] )
//
// Bound by the weights' bytes (half a byte each), so everything is arranged
// around streaming them; no weight is rounded, as each group's sum is scaled in
// fp32.  A word of eight 4-bit weights gives four bf16 pairs by a mask and an
// or each: q | 0x4300 is 128 + q, and 136 less is q - 8, exactly.  The 136 comes off before the
// product: behind it, every partial sum would carry 136 times the row's values and round
// to that, so that an activation of 1e4 on a weight of zero costs a bf16 step.  There are two
// forms: one that shares K out among the
// warps of a block, for calls with so few weight blocks that a block has to take
// little, and one on tensor memory.
#include <cuda_bf16.h>

#include "expert_common.cuh"

namespace a2av {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kSpan = 256;     // K of a TMA box: 128 bytes of a weight row
constexpr int kStages = 4;     // boxes in flight per warp
constexpr int kMaxRows = 32;   // expert rows per work item

// ---- few work items: K shared out among the warps -------------------------------
//
// A block of eight warps takes 16 weight rows; each warp takes every eighth
// span of 256 of K through its own ring of TMA boxes (16 rows x 128 bytes).
// The pairs, less 136, are A fragments of the 16x8x16 matrix instruction,
// whose legacy form is the right one here: the product needs 2 * rows flops
// per weight, far below any tensor limit, and its operands come out of
// registers.  The warps' partial sums meet in shared memory in a fixed order.
// With one row the call is a chain of latencies (launch, places, first box,
// rows, joining): 8.1 us for 21 million weights.  (9.5 with the next item's
// boxes asked for during this one's: two items of a block are rare.)  Loading rows and scales a
// span ahead cost more instructions than it hid (11.7 us).
constexpr int kRows = 16, kBoxBytes = kRows * 128;

struct Shared4 {
    uint64_t full[kWarps][kStages];
    uint32_t abort;
    int32_t warp_sum[kWarps];
};

// Bits i*4 and 16+i*4 of a word: q - 8 of k = 2i and 2i+1 as bf16.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(v) : "r"(w >> (4 * i)));  // (w & mask) | 128.0
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                     __nv_bfloat162{__float2bfloat16(136.0f), __float2bfloat16(136.0f)});
    return *reinterpret_cast<const uint32_t *>(&d);
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory of this form: the warps' rings, their partial sums, the barriers; then the experts' table.
constexpr size_t kSplitParts = (size_t)kWarps * kStages * kBoxBytes;  // offsets
constexpr size_t kSplitShared = kSplitParts + (size_t)kWarps * kRows * (kMaxRows + 1) * 4;
constexpr size_t split_smem_bytes(int E) { return 1024 + kSplitShared + sizeof(Shared4) + (size_t)E * 12; }
static_assert(kSplitShared % 8 == 0 && sizeof(Shared4) % 4 == 0, "alignment");

struct Item {
    int e, row, rows, block;
};

__device__ __forceinline__ Item item_at(long long t, const int32_t *start, const int32_t *count, const int32_t *pre,
                                        int E, int blocks, int most) {
    Item w;
    w.e = expert_of(t, pre, E, blocks);
    const int in = (int)(t - (long long)pre[w.e] * blocks);
    const int chunks = (count[w.e] + most - 1) / most;  // the chunks of one weight block follow each other
    w.block = in / chunks;
    const int first = in % chunks * most;
    w.row = start[w.e] + first;
    w.rows = min(most, count[w.e] - first);
    return w;
}

// One box, 16 weight rows x kSpan of K, for kNT*8 expert rows, into acc.
template <int kNT, bool kSwiglu>
__device__ __forceinline__ void box_sums(const uint32_t *box, const MatmulArgs &a, const Item &w, int k0,
                                         float (&acc)[4][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int words = min(kSpan, a.K - k0) / 32;  // 32-wide steps; K is a multiple of 32
    const int groups = a.K / a.group, per = a.group / 32;
    const uint16_t *x = reinterpret_cast<const uint16_t *>(a.x) + (size_t)w.row * a.K + k0 + t * 8;
    const uint16_t *scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // swiglu: the lower eight rows are gates, the upper eight the same channels' ups
        const int chan = w.block * (kSwiglu ? 8 : 16) + (kSwiglu ? 0 : h * 8) + g;
        const size_t row = (size_t)w.e * a.N * (kSwiglu ? 2 : 1) + (kSwiglu && h ? a.N : 0) + min(chan, a.N - 1);
        scale[h] = static_cast<const uint16_t *>(a.w_scale) + row * groups + k0 / a.group;
    }
    for (int j0 = 0; j0 < words; j0 += per) {  // one group of K at a time
        const float s0 = __uint_as_float((uint32_t)__ldg(scale[0]++) << 16);
        const float s1 = __uint_as_float((uint32_t)__ldg(scale[1]++) << 16);
        float part[kNT][4] = {};
#pragma unroll 4
        for (int j = j0; j < j0 + per; ++j) {
            uint4 b[kNT];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
                b[n] = n * 8 + g < w.rows ? __ldg(reinterpret_cast<const uint4 *>(x + (size_t)(n * 8 + g) * a.K + j * 32))
                                          : make_uint4(0, 0, 0, 0);
            const uint32_t w0 = box[g * 32 + ((j ^ g) * 4 + t)], w1 = box[(8 + g) * 32 + ((j ^ g) * 4 + t)];
            const uint32_t p0 = pair_of(w0, 0), p1 = pair_of(w0, 1), p2 = pair_of(w0, 2), p3 = pair_of(w0, 3);
            const uint32_t q0 = pair_of(w1, 0), q1 = pair_of(w1, 1), q2 = pair_of(w1, 2), q3 = pair_of(w1, 3);
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                mma16816(part[n], p0, q0, p1, q1, b[n].x, b[n].y);
                mma16816(part[n], p2, q2, p3, q3, b[n].z, b[n].w);
            }
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
            acc[n][0] = fmaf(s0, part[n][0], acc[n][0]);
            acc[n][1] = fmaf(s0, part[n][1], acc[n][1]);
            acc[n][2] = fmaf(s1, part[n][2], acc[n][2]);
            acc[n][3] = fmaf(s1, part[n][3], acc[n][3]);
        }
    }
}

template <bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 2) expert_w4_kernel(const __grid_constant__ CUtensorMap map_w,
                                                                const MatmulArgs a) {
    constexpr int kChan = kSwiglu ? kRows / 2 : kRows;  // output channels per work item
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    float *parts = reinterpret_cast<float *>(ring + kSplitParts);  // [warp][kRows][kMaxRows + 1]
    Shared4 *sh = reinterpret_cast<Shared4 *>(ring + kSplitShared);
    const int E = a.g.E;
    int32_t *start = reinterpret_cast<int32_t *>(sh + 1);
    int32_t *count = start + E;
    int32_t *pre = count + E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < kWarps * kStages) mbar_init(&sh->full[tid / kStages][tid % kStages], 1);
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
    uint8_t *mine = ring + warp * kStages * kBoxBytes;
    int put = 0, got = 0;  // boxes issued and consumed
    bool ok = true;
    // (one item a block, unless the splits hold more rows than the plan's tokens make)
    for (long long t = blockIdx.x; t < items; t += gridDim.x) {
        const Item w = item_at(t, start, count, pre, E, blocks, kMaxRows);
        int put_span = warp;
        auto issue = [&] {  // the next box of this warp, if there is one
            if (put_span >= spans) return;
            if (lane == 0) {
                uint64_t *bar = &sh->full[warp][put % kStages];
                mbar_arrive_expect_tx(bar, kBoxBytes);
                asm volatile(
                    "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
                    "%5}], [%6];" ::"r"(smem_u32(mine + put % kStages * kBoxBytes)),
                    "l"(&map_w), "r"(put_span * (kSpan / 8)), "r"(w.block * kChan), "r"(0), "r"(w.e),
                    "r"(smem_u32(bar))
                    : "memory");
            }
            put_span += kWarps;
            ++put;
        };
        for (int i = 0; i < kStages; ++i) issue();
        float acc[4][4] = {};
        for (int span = warp; ok && span < spans; span += kWarps) {
            const int at = got % kStages;
            ok = all_of(mbar_wait_bounded(&sh->full[warp][at], (got / kStages) & 1, a.wait_polls));
            if (!ok) break;
            const uint32_t *box = reinterpret_cast<const uint32_t *>(mine + at * kBoxBytes);
            if (w.rows <= 8) box_sums<1, kSwiglu>(box, a, w, span * kSpan, acc);
            else if (w.rows <= 16) box_sums<2, kSwiglu>(box, a, w, span * kSpan, acc);
            else box_sums<4, kSwiglu>(box, a, w, span * kSpan, acc);
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
        for (int n = 0; n < 4; ++n)
            if (n * 8 < w.rows) {
#pragma unroll
                for (int c = 0; c < 4; ++c) p[((c >> 1) * 8 + g) * (kMaxRows + 1) + n * 8 + q * 2 + (c & 1)] = acc[n][c];
            }
        __syncthreads();
        if (*(volatile uint32_t *)&sh->abort) break;  // the same for every thread: nobody sets it before the next item
        for (int o = tid; o < kChan * w.rows; o += kThreads) {
            const int chan = o % kChan, r = o / kChan;
            float sum = 0.0f, up = 0.0f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                sum += parts[(v * kRows + chan) * (kMaxRows + 1) + r];
                if (kSwiglu) up += parts[(v * kRows + chan + 8) * (kMaxRows + 1) + r];
            }
            const float out = kSwiglu ? swiglu(sum, up) : sum;
            const int n = w.block * kChan + chan;
            if (n < a.N) a.y[(size_t)(w.row + r) * a.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(out));
        }
        __syncthreads();  // the sums are read
    }
    // given up: the boxes that were issued land before the block ends
    for (; got < put; ++got) mbar_wait_bounded(&sh->full[warp][got % kStages], (got / kStages) & 1);
}

// ---- many work items: tensor memory ---------------------------------------------
//
// One persistent block per SM; a work item is 128 weight rows of an expert and up to 16
// of its rows.  Most warps turn the words into bf16 pairs and store them to
// tensor memory, which is where the fifth-generation matrix instruction can
// take its A operand from: lane = weight row, column = two of K, the very
// order in which a word gives its pairs, so a thread reads 16-byte pieces of its own
// row and no unpacked weight touches shared memory.  (At N = 16 the instruction then takes 10
// cycles, against 40 with A in shared memory.)  Each group of K has its own
// accumulator columns, and four warps scale them into fp32 sums in registers.
//
// The steps are short and the way round a buffer is long (barriers and latencies: some
// 2000 cycles for a span of 256 of K, whose weights take 700 to arrive), so
// each buffer has its own four unpacking warps and its own issuing warp (eight
// warps with half a span each: 569 us against 535 on 1,024 rows, the waits
// being per warp), and there are as many buffers as tensor memory holds.  (A
// barrier's parity tells a waiter only that the last phase is over: whoever
// waits for a buffer has to see every phase of it.)  1,024 rows on 256
// experts, K = 7168, SwiGLU to 2048: 540-574 us, 4.4-4.6 TB/s of weights (525-564 with the 136 taken
// off by a second instruction, see above).  No unit is full (256 rows on 32 experts: the ALU pipe 61%, which takes seven of
// an unpacked word's eleven operations, issue 65%, HBM 59%); what is left is the way round a buffer.
constexpr int kMaxCols = 16;                 // expert rows per work item: the instruction's N
constexpr int kACols = kSpan / 2;            // 32-bit columns of a span's A
constexpr int kTileRows = 128;
constexpr int kWBytes = kTileRows * 128, kXBox = kMaxCols * 128, kStage = kWBytes + kSpan / 64 * kXBox;

// For kPer groups of K per 128.
template <int kPer>
struct TmemForm {
    static constexpr int kGroups = 2 * kPer, kDCols = kGroups * kMaxCols;  // of a span
    static constexpr int kBufs = kPer == 1 ? 3 : 2, kStages = kPer == 1 ? 6 : 8;  // (a multiple of the buffers)
    static constexpr int kFirstUnpack = 4, kFirstSum = kFirstUnpack + 4 * kBufs;  // warp 0 loads, 1 .. kBufs issue
    static constexpr int kThreads = (kFirstSum + 4) * 32;
    static_assert(kBufs * (kACols + kDCols) <= 512, "tensor memory");
    static_assert(kStages % kBufs == 0, "every waiter sees every phase of its stages");
};
constexpr int kMaxStages = 8, kMaxBufs = 3;

struct SharedTmem {
    uint64_t full[kMaxStages], empty[kMaxStages];
    // ready: a half of A is filled (and the accumulators of a round ago are read); done: the instructions have ended
    uint64_t ready[2][kMaxBufs], done[kMaxBufs], drain;
    uint32_t tmem, abort;
    int32_t warp_sum[32];
};
constexpr size_t tmem_shared(int stages) { return (size_t)stages * kStage; }  // offset behind the stages
constexpr size_t tmem_smem_bytes(int stages, int E) {
    return 1024 + tmem_shared(stages) + sizeof(SharedTmem) + (size_t)E * 12;
}
static_assert(kStage % 1024 == 0 && tmem_smem_bytes(kMaxStages, kMaxExperts) <= 232448, "shared memory");

// A position in a ring of n buffers and the parity of its current round.
struct Ring {
    int i = 0;
    uint32_t parity;
    __device__ explicit Ring(uint32_t p) : parity(p) {}
    __device__ __forceinline__ void next(int n, int steps = 1) {
        i += steps;
        if (i >= n) {
            i -= n;
            parity ^= 1;
        }
    }
};

// Eight weights of a word as four bf16 pairs, k ascending.
__device__ __forceinline__ void unpack_word(uint32_t w, uint32_t *p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pair_of(w, i);
}

// The bf16 scales of groups at .. at + kGroups - 1 of a weight row, in pairs; zeros behind the last. In one load
// where they lie aligned: the lanes' rows are apart, and each load of a warp takes a cycle per row.
template <int kGroups>
__device__ __forceinline__ void fetch_scales(uint32_t (&to)[kGroups / 2], const uint16_t *from, int at, int groups,
                                             bool aligned) {
#pragma unroll
    for (int i = 0; i < kGroups / 2; ++i) to[i] = 0;
    if (at >= groups) return;
    if (aligned) {
        if constexpr (kGroups == 2) {
            to[0] = __ldg(reinterpret_cast<const uint32_t *>(from + at));
        } else if constexpr (kGroups == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(from + at));
            to[0] = v.x, to[1] = v.y;
        } else {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(from + at));
            to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
        if (at + i < groups) to[i / 2] |= (uint32_t)__ldg(from + at + i) << (i % 2 * 16);
}

// acc[n] += scale[i] * D_i[n] for the first kCols rows, kAtMost groups' columns at a time.
template <int kCols, int kAtMost, int kGroups>
__device__ __forceinline__ void add_groups(uint32_t d, const float (&scale)[kGroups], float (&acc)[kMaxCols]) {
    constexpr int kAtOnce = kGroups < kAtMost ? kGroups : kAtMost;
#pragma unroll
    for (int i0 = 0; i0 < kGroups; i0 += kAtOnce) {
        float v[kAtOnce][kCols];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) tmem_ld<kCols>(d + (i0 + i) * kMaxCols, v[i]);
        tmem_wait_ld(v);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
            for (int n = 0; n < kCols; ++n) acc[n] = fmaf(scale[i0 + i], v[i][n], acc[n]);
    }
}

template <bool kSwiglu, int kPer>
__global__ void __launch_bounds__(TmemForm<kPer>::kThreads, 1)
    expert_w4_tmem_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                          const MatmulArgs a) {
    using F = TmemForm<kPer>;
    constexpr int kChan = kSwiglu ? kTileRows / 2 : kTileRows;  // output channels per item
    constexpr int kBufs = F::kBufs, kDCols = F::kDCols, kGroups = F::kGroups;
    extern __shared__ uint8_t raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    SharedTmem *sh = reinterpret_cast<SharedTmem *>(stages + tmem_shared(F::kStages));
    const int E = a.g.E;
    int32_t *start = reinterpret_cast<int32_t *>(sh + 1);
    int32_t *count = start + E;
    int32_t *pre = count + E;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), quad = warp & 3;
    if (tid == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 5);  // the four warps that read its words, and the instructions that read its rows
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sh->ready[0][i], 8);  // four warps fill, four read
            mbar_init(&sh->ready[1][i], 4);
            mbar_init(&sh->done[i], 1);
        }
        mbar_init(&sh->drain, kBufs);
        sh->abort = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w));
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_x));
    }
    grid_dependency_wait();
    // Tensor memory is taken after the wait: the kernel before may take its own late, and this one may start early.
    if (warp == 1) tmem_alloc_all(&sh->tmem);
    tmem_fence_before();
    const int total = place_experts<F::kThreads>(a, kMaxCols, start, count, pre, sh->warp_sum);  // ends in a barrier
    tmem_fence_after();
    const uint32_t tmem = sh->tmem, d0 = tmem + kBufs * kACols;
    const int blocks = (a.N + kChan - 1) / kChan;
    const long long items = (long long)total * blocks;
    const int spans = (a.K + kSpan - 1) / kSpan;
    // spans of this block, all items (what lies past K is zero in x)
    const long long mine = (long long)blockIdx.x < items ? ((items - 1 - blockIdx.x) / gridDim.x + 1) * spans : 0;
    const long long polls = a.wait_polls;

    if (warp == 0) {
        Ring s(1);
        uint32_t fills = 0;
        bool ok = true;
        for (long long t = blockIdx.x; ok && t < items; t += gridDim.x) {
            const Item w = item_at(t, start, count, pre, E, blocks, kMaxCols);
            const int row = __shfl_sync(0xffffffffu, w.row, 0), e = __shfl_sync(0xffffffffu, w.e, 0),
                      block = __shfl_sync(0xffffffffu, w.block, 0);
            for (int span = 0; span < spans; ++span) {
                ok = all_of(wait_or_abort(&sh->empty[s.i], s.parity, polls, &sh->abort, a.status));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t at = smem_u32(stages) + s.i * kStage;
                    uint64_t *bar = &sh->full[s.i];
                    mbar_arrive_expect_tx(bar, kStage);
                    asm volatile(
                        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
                        "%3, %3, %4, %5}], [%6];" ::"r"(at),
                        "l"(&map_w), "r"(span * (kSpan / 8)), "r"(0), "r"(block * (kChan / 8)), "r"(e),
                        "r"(smem_u32(bar))
                        : "memory");
#pragma unroll
                    for (int i = 0; i < kSpan / 64; ++i)
                        asm volatile(
                            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
                            "{%2, %3}], [%4];" ::"r"(at + kWBytes + i * kXBox),
                            "l"(&map_x), "r"(span * kSpan + i * 64), "r"(row), "r"(smem_u32(bar))
                            : "memory");
                }
                __syncwarp();
                s.next(F::kStages);
                ++fills;
            }
        }
        // every load that was issued lands before the block ends, also if other warps gave up
        for (int i = 0; i < F::kStages && fills > 0; ++i, --fills) {
            if (--s.i < 0) {
                s.i = F::kStages - 1;
                s.parity ^= 1;
            }
            mbar_wait_bounded(&sh->full[s.i], s.parity ^ 1);
        }
    } else if (warp <= kBufs) {
        constexpr uint32_t kIdesc =
            1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(kMaxCols >> 3) << 17 | (uint32_t)(kTileRows >> 4) << 24;
        constexpr int kSteps = kSpan / 16, kPerGroup = kSteps / kGroups;
        const int b = warp - 1;
        const uint32_t at = tmem + b * kACols, d = d0 + b * kDCols;
        Ring s(0);
        s.i = b;
        uint32_t parity = 0;
        for (long long c = b; c < mine; c += kBufs) {
            bool ok = all_of(wait_or_abort(&sh->full[s.i], s.parity, polls, &sh->abort, a.status));  // the rows
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // the first half's instructions run while the second is unpacked
                ok = ok && all_of(wait_or_abort(&sh->ready[half][b], parity, polls, &sh->abort, a.status));
                if (!ok) break;
                tmem_fence_after();
                if (elect_one()) {
                    const uint32_t rows = smem_u32(stages) + s.i * kStage + kWBytes;
#pragma unroll
                    for (int j = half * (kSteps / 2); j < (half + 1) * (kSteps / 2); ++j) {
                        const uint64_t bd = operand_desc(rows + j / 4 * kXBox) + j % 4 * 2;
                        mma_tmem(d + j / kPerGroup * kMaxCols, at + j * 8, bd, kIdesc, j % kPerGroup != 0);
                    }
                    if (half == 1) {
                        mma_commit_one(&sh->done[b]);
                        mma_commit_one(&sh->empty[s.i]);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
            parity ^= 1;
            s.next(F::kStages, kBufs);
        }
        // the instructions that were issued end before tensor memory is freed
        if (elect_one()) mma_commit_one(&sh->drain);
        mbar_wait_bounded(&sh->drain, 0);
    } else if (warp >= F::kFirstSum) {
        const int groups = a.K / a.group;
        const bool up = kSwiglu && (lane & 8);
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const bool aligned = groups % kGroups == 0 && reinterpret_cast<uintptr_t>(a.w_scale) % 16 == 0;
        Ring buf(0);
        bool ok = true;
        if (lane == 0)
            for (int i = 0; i < kBufs; ++i) mbar_arrive(&sh->ready[0][i]);  // nothing to read in the first round
        for (long long t = blockIdx.x; ok && t < items; t += gridDim.x) {
            const Item w = item_at(t, start, count, pre, E, blocks, kMaxCols);
            // swiglu: lanes 0-7 gate of channels 0-7, 8-15 their up, 16-23 gate of channels 8-15, ...
            const int chan =
                w.block * kChan + (kSwiglu ? quad * 16 + (lane >> 4) * 8 + (lane & 7) : quad * 32 + lane);
            const size_t row = (size_t)w.e * a.N * (kSwiglu ? 2 : 1) + (up ? a.N : 0) + min(chan, a.N - 1);
            const uint16_t *from = static_cast<const uint16_t *>(a.w_scale) + row * groups;
            float acc[kMaxCols] = {};
            uint32_t next[kGroups / 2];
            fetch_scales<kGroups>(next, from, 0, groups, aligned);
            for (int c = 0; c < spans; ++c) {
                float scale[kGroups];
#pragma unroll
                for (int i = 0; i < kGroups; i += 2) {
                    scale[i] = __uint_as_float(next[i / 2] << 16);
                    scale[i + 1] = __uint_as_float(next[i / 2] & 0xffff0000u);
                }
                // the next span's scales while this one's sums are waited for
                fetch_scales<kGroups>(next, from, (c + 1) * kGroups, groups, aligned);
                ok = all_of(wait_or_abort(&sh->done[buf.i], buf.parity, polls, &sh->abort, a.status));
                if (!ok) break;
                tmem_fence_after();
                // (with two groups a span there is little to leave out, and registers are few)
                const uint32_t d = d0 + lanes + buf.i * kDCols;
                if (kPer == 1) add_groups<16, 1>(d, scale, acc);
                else if (w.rows <= 4) add_groups<4, 8>(d, scale, acc);
                else if (w.rows <= 8) add_groups<8, 4>(d, scale, acc);
                else add_groups<16, 2>(d, scale, acc);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->ready[0][buf.i]);
                buf.next(kBufs);
            }
            if (!ok) break;
            uint16_t *y = a.y + (size_t)w.row * a.N + chan;
            if (kSwiglu) {
                // of rows n, n+1 the gate lane finishes the first, the up lane the second
#pragma unroll
                for (int n = 0; n < kMaxCols; n += 2) {
                    const float other = __shfl_xor_sync(0xffffffffu, up ? acc[n] : acc[n + 1], 8);
                    const float g = up ? other : acc[n], u = up ? acc[n + 1] : other;
                    const int r = n + (up ? 1 : 0);
                    const float out = swiglu(g, u);
                    if (chan < a.N && r < w.rows)
                        y[(size_t)r * a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(out));
                }
            } else if (chan < a.N) {
#pragma unroll
                for (int n = 0; n < kMaxCols; ++n)
                    if (n < w.rows) y[(size_t)n * a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[n]));
            }
        }
    } else if (warp >= F::kFirstUnpack) {
        // this warp's lanes: weight rows quad*32 + lane of every kBufs-th span
        const int b = (warp - F::kFirstUnpack) >> 2, row = quad * 32 + lane;
        const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + b * kACols;
        Ring s(0);
        s.i = b;
        uint32_t parity = 1;
        for (long long c = b; c < mine; c += kBufs) {
            if (!all_of(wait_or_abort(&sh->full[s.i], s.parity, polls, &sh->abort, a.status)) ||
                !all_of(wait_or_abort(&sh->done[b], parity, polls, &sh->abort, a.status)))
                break;
            tmem_fence_after();
            const uint8_t *words = stages + s.i * kStage + row * 128;
#pragma unroll
            for (int h = 0; h < 4; ++h) {  // 64 of K: 32 columns
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(words + (((h * 2 + i) ^ (row & 7)) << 4));
                    unpack_word(v.x, p + i * 16);
                    unpack_word(v.y, p + i * 16 + 4);
                    unpack_word(v.z, p + i * 16 + 8);
                    unpack_word(v.w, p + i * 16 + 12);
                }
                tmem_st32(to + h * 32, p);
                if (h == 3) {
                    __syncwarp();  // every lane has its words
                    if (lane == 0) mbar_arrive(&sh->empty[s.i]);
                }
                if (h % 2 == 1) {
                    tmem_wait_st();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->ready[h / 2][b]);
                }
            }
            parity ^= 1;
            s.next(F::kStages, kBufs);
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (warp == 1) {
        tmem_fence_after();
        tmem_free_all(tmem);
    }
}

template <bool kSwiglu, int kPer>
cudaError_t launch_w4_tmem(const a2av_plan_s &p, const MatmulArgs &a, cudaStream_t s) {
    constexpr int kChan = kSwiglu ? kTileRows / 2 : kTileRows;
    const cuuint64_t halves = kSwiglu ? 2 : 1, row = (cuuint64_t)a.K / 2, N = a.N;
    CUtensorMap mw, mx;
    // w as [E][N/8][gate, up][8][K/8]
    const cuuint64_t wd[5] = {(cuuint64_t)a.K / 8, 8, halves, N / 8, (cuuint64_t)a.g.E};
    const cuuint64_t wst[4] = {row, N * row, 8 * row, halves * N * row};
    const cuuint32_t wb[5] = {kSpan / 8, 8, (cuuint32_t)halves, kChan / 8, 1};
    const cuuint64_t xd[2] = {(cuuint64_t)a.K, (cuuint64_t)a.arena_rows}, xst[1] = {(cuuint64_t)a.x_pitch};
    const cuuint32_t xb[2] = {64, kMaxCols};
    if (!encode_map(&mw, CU_TENSOR_MAP_DATA_TYPE_INT32, 5, a.w, wd, wst, wb) ||
        !encode_map(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.x, xd, xst, xb))
        return cudaErrorInvalidValue;
    const auto kernel = expert_w4_tmem_kernel<kSwiglu, kPer>;
    const size_t smem = tmem_smem_bytes(TmemForm<kPer>::kStages, a.g.E);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e =
        allow_smem(kernel, allowed, p.cfg.device, tmem_smem_bytes(TmemForm<kPer>::kStages, kMaxExperts));
    if (e != cudaSuccess) return e;
    const long long rows = a.rows_most;
    const long long most = ((rows < a.g.E ? rows : a.g.E) + rows / kMaxCols) * ((a.N + kChan - 1) / kChan);
    return launch_pdl(kernel, (int)(most < p.num_sms ? most : p.num_sms), TmemForm<kPer>::kThreads, smem, s, mw, mx, a);
}

template <bool kSwiglu>
cudaError_t launch_w4_groups(const a2av_plan_s &p, const MatmulArgs &a, cudaStream_t s) {
    return a.group == 32   ? launch_w4_tmem<kSwiglu, 4>(p, a, s)
           : a.group == 64 ? launch_w4_tmem<kSwiglu, 2>(p, a, s)
                           : launch_w4_tmem<kSwiglu, 1>(p, a, s);
}

// the most items of the split form that the call's rows can make
long long split_items(const MatmulArgs &a, bool swiglu) {
    const long long rows = a.rows_most, chans = swiglu ? kRows / 2 : kRows;
    return ((rows < a.g.E ? rows : a.g.E) + rows / kMaxRows) * ((a.N + chans - 1) / chans);
}

template <bool kSwiglu>
cudaError_t launch_w4_split(const a2av_plan_s &p, const MatmulArgs &a, cudaStream_t s) {
    constexpr int kChan = kSwiglu ? kRows / 2 : kRows;
    const cuuint64_t halves = kSwiglu ? 2 : 1, row = (cuuint64_t)a.K / 2;
    CUtensorMap m;
    // w as [E][gate, up][N][K/8]
    const cuuint64_t dims[4] = {(cuuint64_t)a.K / 8, (cuuint64_t)a.N, halves, (cuuint64_t)a.g.E};
    const cuuint64_t strides[3] = {row, a.N * row, halves * a.N * row};
    const cuuint32_t box[4] = {kSpan / 8, kChan, (cuuint32_t)halves, 1};
    if (!encode_map(&m, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, a.w, dims, strides, box)) return cudaErrorInvalidValue;
    const size_t smem = split_smem_bytes(a.g.E);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(expert_w4_kernel<kSwiglu>, allowed, p.cfg.device, split_smem_bytes(kMaxExperts));
    if (e != cudaSuccess) return e;
    // (the caller has seen to it that so many blocks fit at once)
    return launch_pdl(expert_w4_kernel<kSwiglu>, (int)split_items(a, kSwiglu), kThreads, smem, s, m, a);
}

}  // namespace

cudaError_t launch_expert_w4(const a2av_plan_s &p, const MatmulArgs &a, bool swiglu, cudaStream_t s) {
    // The split form while all its items (16 weight rows each) are resident at once, two to an SM; when some would have
    // to wait for a turn the form on tensor memory is the faster one.  One row to 4096 (256 items): K = 2048 5.9 us
    // split, 8.3 on tensor memory, 4096 8.6 and 12.2, 8192 14.1 and 20.3; to 5120 (320 items), K = 2048: 9.7 and 8.3;
    // to 6144: K = 1024 8.9 and 6.2, 8192 25 and 20.  K = 5120, SwiGLU to 2048: one expert 8.1 and 13.0, two 15.3 and
    // 13.3, sixteen 93 and 37.
    if (split_items(a, swiglu) > 2 * p.num_sms)
        return swiglu ? launch_w4_groups<true>(p, a, s) : launch_w4_groups<false>(p, a, s);
    return swiglu ? launch_w4_split<true>(p, a, s) : launch_w4_split<false>(p, a, s);
}

}  // namespace a2av
