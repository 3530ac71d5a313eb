// The experts' products on the dispatched rows, bf16 or e4m3 (tcgen05):
//
//   y[r][n] = act( sum_k x[r][k] * w[e(r)][n][k] ),  the rows of expert e = rows [start_e, start_e + count_e)
//
// with start and count read on the device from the split arrays.  The weights
// are the M side of the matrix instruction (256 rows per tile) and an
// expert's rows the N side: N may be any multiple of 32 up to 256, so a group
// of c rows costs ceil(c/32)*32 columns, not a multiple of 128, and a group of
// a few rows streams the weights once with a narrow instruction.  Many rows:
// bound by the tensor pipe (90% active; 8 x 1,024 rows, 5120 -> 2 x 2048: 195-205 us,
// 1.68-1.76 PFLOP/s); few: by the weights' bytes (16 rows over 16 experts, about
// ten of them live: 76 us, 420 MB at 5.5 TB/s).
//
// One persistent pair of blocks per two SMs (a cluster, cta_group::2): each
// block loads its 128 of the tile's 256 weight rows and half of its expert
// rows, and the instruction reads both halves of the latter out of the two
// shared memories.  In each block warp 0 feeds a ring of stages by TMA; warp 1 of the
// first block issues the instructions into one of two TMEM accumulators;
// warps 2-9 drain the other one (lane = channel, column = row), apply scales
// and activation in fp32 and store bf16.
//
// SwiGLU: a block's tile holds the gate and the up weights of 64 channels in
// alternating blocks of eight rows (one TMA box of a five-dimensional view
// of w), so the two halves of a channel sit eight TMEM lanes apart in the
// same warp: one shuffle per two rows brings them together.
#include <cuda_bf16.h>
#include <stddef.h>

#include "expert_common.cuh"

namespace a2av {
namespace {

constexpr int kEpiWarps = 8;        // two for each quarter of the TMEM lanes
constexpr int kThreads = 64 + kEpiWarps * 32;  // after the producer warp and the matrix warp
constexpr int kStages = 6;
constexpr int kRowBytes = 128;      // K bytes per stage row: one 128-byte swizzle span
constexpr int kTileM = 128;         // weight rows per block of a pair
constexpr int kTileN = 256;         // expert rows per tile, at most
constexpr int kABytes = kTileM * kRowBytes;
constexpr int kBBytes = kTileN / 2 * kRowBytes;  // half of them in each block
// The ring: six stages for any tile; or, when no expert has more than 32 rows, ten whose row part holds just these:
// such a call streams weights, and what an SM gets is what it has in flight (16 rows over 16 experts: 76 us
// against 83 with the six).
constexpr int kStageBytes = kABytes + kBBytes, kRingBytes = kStages * kStageBytes;
constexpr int kFewRows = 32, kFewStageBytes = kABytes + kFewRows / 2 * kRowBytes, kFewStages = 10;
static_assert(kFewStages * kFewStageBytes <= kRingBytes && kFewStageBytes % 1024 == 0, "one ring");
// Rows of x a block loads at once: the first box that holds its share (128 at most).
__host__ __device__ constexpr int box_rows(int i) { return i == 0 ? 16 : i == 1 ? 64 : 128; }
constexpr int kBand = 8;            // row tiles of an expert that run with one channel tile in turn

struct Shared {
    uint64_t full[kFewStages], empty[kFewStages];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    uint32_t abort;
    uint32_t other_fills;  // of the ring, by the other block
    int32_t warp_sum[kThreads / 32];
    alignas(16) float x_scale[kEpiWarps][kTileN / 2];  // of the expert rows an epilogue warp takes
};

static_assert(sizeof(Shared) % 16 == 0 && offsetof(Shared, x_scale) % 16 == 0, "the scales are read four at a time");

template <bool kFp8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    const uint32_t acc = accumulate ? 1u : 0u;
    if (kFp8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
// Arrives on `bar` of this block, or of both blocks of the pair, once the instructions issued so far are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void mma_commit_both(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// The address of this block's shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(const void *p, uint32_t rank) {
    uint32_t d;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(p)), "r"(rank));
    return d;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Loads into this block's shared memory that count on a barrier of the pair's first block (`bar`).
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *m, int k, int row, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(m), "r"(k), "r"(row), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_weights(uint32_t dst, const CUtensorMap *m, int k, int block, int e, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%3, %4, %5}], [%6];" ::"r"(dst),
        "l"(m), "r"(k), "r"(0), "r"(block), "r"(e), "r"(bar)
        : "memory");
}

struct RowMaps {
    CUtensorMap box[3];
};
// Boxes a call can use: counts are cut to the arena, and an expert of up to kFewRows rows needs the first alone.
__host__ __device__ inline int row_boxes(const MatmulArgs &a) { return a.arena_rows > kFewRows ? 3 : 1; }

// One unit of work: rows [row, row + rows) of expert e times channel tile `ctile`.
struct Tile {
    int e, row, rows, ctile;
};

__device__ __forceinline__ Tile tile_at(long long t, const int32_t *start, const int32_t *count, const int32_t *pre,
                                        int E, int ctiles) {
    const int lo = expert_of(t, pre, E, ctiles);
    const int n = count[lo];
    const int rt = (n + kTileN - 1) / kTileN;
    // An expert's row tiles are taken kBand at a time, every channel tile of
    // a band before the next band: the band's rows and the weights stay in L2
    // while they are used again.
    const long long in = t - (long long)pre[lo] * ctiles;
    const int band = (int)(in / (kBand * ctiles));
    const int wide = min(kBand, rt - band * kBand);
    const int rem = (int)(in - (long long)band * kBand * ctiles);
    Tile r;
    r.e = lo;
    r.ctile = rem / wide;
    // even shares, multiples of 32 rows; the last one takes what is left, which is a row at least: rounding up adds at
    // most 31 rows to a share, and nothing to the share of more than seven tiles (their mean is above 224, share 256)
    const int share = ((n + rt - 1) / rt + 31) / 32 * 32;
    const int first = (band * kBand + rem % wide) * share;
    r.row = start[lo] + first;
    r.rows = min(share, n - first);
    return r;
}

__device__ __forceinline__ Tile uniform(const Tile &t) {
    return Tile{__shfl_sync(0xffffffffu, t.e, 0), __shfl_sync(0xffffffffu, t.row, 0), __shfl_sync(0xffffffffu, t.rows, 0),
                __shfl_sync(0xffffffffu, t.ctile, 0)};
}

// Shared memory: the ring, the barriers, the experts' table.
constexpr size_t smem_bytes(int E) { return 1024 + kRingBytes + sizeof(Shared) + (size_t)E * 12; }
static_assert(smem_bytes(kMaxExperts) <= 232448, "shared memory");

template <bool kFp8, bool kSwiglu>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_x,
                       const MatmulArgs a) {
    extern __shared__ uint8_t raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Shared *sh = reinterpret_cast<Shared *>(stages + kRingBytes);
    const int E = a.g.E;
    int32_t *start = reinterpret_cast<int32_t *>(sh + 1);
    int32_t *count = start + E;
    int32_t *pre = count + E;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = blockIdx.x & 1;  // in the pair (the cluster's dimension is two)
    const uint32_t peer_abort = in_block(&sh->abort, rank ^ 1);

    if (tid == 0) {
        for (int s = 0; s < kFewStages; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh->acc_full[b], 1);
            mbar_init(&sh->acc_empty[b], 2 * kEpiWarps);
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
    }
    if (tid == 64) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w));
        for (int i = 0; i < row_boxes(a); ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(&map_x.box[i]));
    }
    grid_dependency_wait();

    // Tensor memory is taken after the wait: the kernel before may take its own late, and this one may start early.
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tmem_fence_before();
    const int total = place_experts<kThreads>(a, kTileN, start, count, pre, sh->warp_sum);  // ends in a barrier
    bool more_rows = false;
    for (int e = tid; e < E; e += kThreads) more_rows |= count[e] > kFewRows;
    more_rows = __syncthreads_or(more_rows);
    const int ring = more_rows ? kStages : kFewStages, stage_bytes = more_rows ? kStageBytes : kFewStageBytes;
    cluster_sync();  // the other block's barriers are set up, too
    tmem_fence_after();

    const uint32_t tmem = sh->tmem;
    constexpr int kChan = kSwiglu ? kTileM / 2 : kTileM;  // output channels per block
    const int ctiles = (a.N + 2 * kChan - 1) / (2 * kChan);
    const long long tiles = (long long)total * ctiles;
    constexpr int kStep = kFp8 ? kRowBytes : kRowBytes / 2;  // K elements per stage
    const int kblocks = (a.K + kStep - 1) / kStep;

    // Where the loads stand (warp 0): tile, K block, stage, the parity that
    // says a stage is free, and how many fills were issued.
    long long put_t = blockIdx.x / 2;
    int put_kb = 0, put_s = 0;
    uint32_t put_parity = 1, fills = 0;
    const uint32_t base = smem_u32(stages), full0 = in_block(&sh->full[0], 0);
    // Issues fills as stages come free, until the end (true) or a give-up; or, without waiting, until
    // `until` were issued.  The whole warp runs the loop and one elected lane issues, so that the
    // instructions' operands are uniform registers; the next stage's barrier is looked at before the
    // loads are issued, so that its answer is there afterwards.
    auto produce = [&](bool wait, uint32_t until) {
        bool free = false;
        for (; put_t < tiles; put_t += gridDim.x / 2, put_kb = 0) {
            const Tile w = uniform(tile_at(put_t, start, count, pre, E, ctiles));
            const int half = (w.rows + 31) / 32 * 16;  // expert rows per block
            const int row = w.row + rank * half, block = (w.ctile * 2 + rank) * (kChan / 8);
            const int box = half <= box_rows(0) ? 0 : half <= box_rows(1) ? 1 : 2;
            const CUtensorMap *const map = &map_x.box[box];
            const uint32_t bytes = 2 * (kABytes + box_rows(box) * kRowBytes);
            for (; put_kb < kblocks; ++put_kb) {
                if (!wait ? (int32_t)(until - fills) <= 0
                          : !free && !all_of(wait_or_abort(&sh->empty[put_s], put_parity, a.wait_polls, &sh->abort,
                                                           a.status, peer_abort)))
                    return false;
                const int s = put_s;
                if (++put_s == ring) {
                    put_s = 0;
                    put_parity ^= 1;
                }
                free = wait && a.wait_polls > 0 && mbar_test_wait(&sh->empty[put_s], put_parity);
                if (elect_one()) {
                    const uint32_t at = base + s * stage_bytes, bar = full0 + s * 8;
                    if (rank == 0) mbar_arrive_expect_tx(&sh->full[s], bytes);
                    tma_weights(at, &map_w, put_kb * kStep, block, w.e, bar);
                    tma_rows(at + kABytes, map, put_kb * kStep, row, bar);
                }
                __syncwarp();
                free = all_of(free);
                ++fills;
            }
        }
        return true;
    };

    if (warp == 0) {
        bool ok = produce(true, 0);
        // the arrivals on the last fills' barriers come from the first block: they are in before this one may end
        for (int i = 0, s = put_s, par = put_parity; ok && i < ring; ++i) {
            ok = all_of(wait_or_abort(&sh->empty[s], par, a.wait_polls, &sh->abort, a.status, peer_abort));
            if (++s == ring) {
                s = 0;
                par ^= 1;
            }
        }
        // how far this block got, for the other one if the pair gives up
        if (lane == 0)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_block(&sh->other_fills, rank ^ 1)), "r"(fills)
                         : "memory");
    } else if (warp == 1) {
        if (rank == 0) {
            // fp32 accumulator; A and B bf16 (1) or e4m3 (0), both K-major; M of the pair
            constexpr uint32_t kIdesc = 1u << 4 | (kFp8 ? 0u : 1u << 7 | 1u << 10) | (uint32_t)(2 * kTileM >> 4) << 24;
            int s = 0, b = 0;
            uint32_t parity = 0, acc_parity = 1;
            bool ok = true, in = false;
            for (long long t = blockIdx.x / 2; ok && t < tiles; t += gridDim.x / 2) {
                const int rows = uniform(tile_at(t, start, count, pre, E, ctiles)).rows;
                ok = all_of(wait_or_abort(&sh->acc_empty[b], acc_parity, a.wait_polls, &sh->abort, a.status, peer_abort));
                tmem_fence_after();
                const uint32_t idesc = kIdesc | (uint32_t)((rows + 31) / 32 * 4) << 17, d = tmem + b * kTileN;
                for (int kb = 0; ok && kb < kblocks; ++kb) {
                    ok = in || all_of(wait_or_abort(&sh->full[s], parity, a.wait_polls, &sh->abort, a.status, peer_abort));
                    if (!ok) break;
                    const int now = s;
                    if (++s == ring) {
                        s = 0;
                        parity ^= 1;
                    }
                    in = mbar_test_wait(&sh->full[s], parity);
                    tmem_fence_after();
                    if (elect_one()) {
                        const uint32_t at = base + now * stage_bytes;
                        const uint64_t da = operand_desc(at), db = operand_desc(at + kABytes);
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // 32 bytes of K per instruction
                            mma<kFp8>(d, da + j * 2, db + j * 2, idesc, kb > 0 || j > 0);
                        mma_commit_both(&sh->empty[now]);
                        if (kb == kblocks - 1) mma_commit_both(&sh->acc_full[b]);
                    }
                    __syncwarp();
                    in = all_of(in);
                }
                b ^= 1;
                if (b == 0) acc_parity ^= 1;
            }
            // every instruction that was issued ends before TMEM is freed, also where an epilogue gave up
            if (elect_one()) mma_commit(&sh->drain);
            mbar_wait_bounded(&sh->drain, 0);
        }
    } else {
        // 32 columns at a time, the two warps of a quarter in turn
        const int quad = warp & 3, side = (warp - 2) >> 2;
        float *const scales = sh->x_scale[warp - 2];
        uint32_t it = 0;
        const bool up = kSwiglu && (lane & 8);
        for (long long t = blockIdx.x / 2; t < tiles; t += gridDim.x / 2, ++it) {
            const Tile w = tile_at(t, start, count, pre, E, ctiles);
            const int b = it & 1;
            // swiglu: lanes 0-7 gate of channels 0-7, 8-15 their up, 16-23 gate of channels 8-15, ...
            const int chan = (w.ctile * 2 + rank) * kChan +
                             (kSwiglu ? quad * 16 + (lane >> 4) * 8 + (lane & 7) : quad * 32 + lane);
            const bool store = chan < a.N;
            float ws = 1.0f;
            if (kFp8) {
                if (store)
                    ws = __ldg(static_cast<const float *>(a.w_scale) + (size_t)w.e * a.N * (kSwiglu ? 2 : 1) +
                               (up ? a.N : 0) + chan);
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // the rows' scales, behind their values
                    const int r = i * 64 + side * 32 + lane;
                    if (r < w.rows)
                        scales[i * 32 + lane] =
                            __ldg(reinterpret_cast<const float *>(a.x + (size_t)(w.row + r) * a.x_pitch + a.K));
                }
                __syncwarp();
            }
            if (!all_of(wait_or_abort(&sh->acc_full[b], (it >> 1) & 1, a.wait_polls, &sh->abort, a.status, peer_abort)))
                break;
            tmem_fence_after();
            uint16_t *y = a.y + (size_t)w.row * a.N + chan;
            for (int c = side * 32; c < w.rows; c += 64) {
                float got[1][32];
                tmem_ld<32>(tmem + ((uint32_t)(quad * 32) << 16) + b * kTileN + c, got[0]);
                tmem_wait_ld(got);
                float(&v)[32] = got[0];
                if (kFp8) {
                    const float4 *xs = reinterpret_cast<const float4 *>(scales + (c >> 6) * 32);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 x4 = xs[i];
                        v[i * 4] *= ws * x4.x;
                        v[i * 4 + 1] *= ws * x4.y;
                        v[i * 4 + 2] *= ws * x4.z;
                        v[i * 4 + 3] *= ws * x4.w;
                    }
                }
                if (kSwiglu) {
                    // of rows i, i+1 the gate lane finishes the first, the up lane the second
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 1], 8);
                        const float g = up ? other : v[i], u = up ? v[i + 1] : other;
                        const int row = c + i + (up ? 1 : 0);
                        const float out = swiglu(g, u);
                        if (store && row < w.rows)
                            y[(size_t)row * a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(out));
                    }
                } else if (store) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i < w.rows)
                            y[(size_t)(c + i) * a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0)  // the first block issues
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                 in_block(&sh->acc_empty[b], 0))
                             : "memory");
        }
    }
    __syncwarp();
    tmem_fence_before();
    cluster_sync();  // both blocks are done with the other's shared memory and with TMEM
    if (*(volatile uint32_t *)&sh->abort) {
        // Given up (both blocks know: the flag is set in both before this
        // barrier).  The block that is behind issues the loads the other has
        // issued, so that every fill is whole, and the first block waits for
        // them to land: the last fill of each stage.  And the second block waits
        // for what the first one's instructions still send to its barriers: one
        // more arrival, behind theirs.
        if (warp == 0) {
            produce(false, *(volatile uint32_t *)&sh->other_fills);
            for (int i = 0; rank == 0 && i < ring; ++i) {
                if (--put_s < 0) {
                    put_s = ring - 1;
                    put_parity ^= 1;
                }
                if (fills-- > 0) mbar_wait_bounded(&sh->full[put_s], put_parity ^ 1);
                else break;
            }
        } else if (warp == 1) {
            if (rank == 0 && elect_one()) mma_commit_both(&sh->drain);
            mbar_wait_bounded(&sh->drain, rank ^ 1);  // the first block's second phase, the other's first
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp == 1) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <bool kFp8, bool kSwiglu>
cudaError_t launch_gemm(const a2av_plan_s &p, const MatmulArgs &a, cudaStream_t s) {
    const cuuint64_t es = kFp8 ? 1 : 2, K = a.K, N = a.N, E = a.g.E, halves = kSwiglu ? 2 : 1;
    const cuuint32_t step = kRowBytes / (cuuint32_t)es;
    CUtensorMap mw;
    RowMaps mx{};
    // w as [E][N/8][gate, up][8][K]
    const cuuint64_t wd[5] = {K, 8, halves, N / 8, E};
    const cuuint64_t wst[4] = {K * es, N * K * es, 8 * K * es, halves * N * K * es};
    const cuuint32_t wb[5] = {step, 8, (cuuint32_t)halves, (cuuint32_t)(kTileM / 8 / halves), 1};
    const cuuint64_t xd[2] = {K, (cuuint64_t)a.arena_rows};
    const cuuint64_t xst[1] = {(cuuint64_t)a.x_pitch};
    const CUtensorMapDataType type = kFp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!encode_map(&mw, type, 5, a.w, wd, wst, wb)) return cudaErrorInvalidValue;
    for (int i = 0; i < row_boxes(a); ++i) {
        const cuuint32_t xb[2] = {step, (cuuint32_t)box_rows(i)};
        if (!encode_map(&mx.box[i], type, 2, a.x, xd, xst, xb)) return cudaErrorInvalidValue;
    }
    const size_t smem = smem_bytes(a.g.E);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e =
        allow_smem(expert_gemm_kernel<kFp8, kSwiglu>, allowed, p.cfg.device, smem_bytes(kMaxExperts));
    if (e != cudaSuccess) return e;
    // at most this many tiles: each expert with rows begins one more than its rows fill
    const long long rows = a.rows_most, chan = kSwiglu ? kTileM : 2 * kTileM;
    const long long most = ((rows < (long long)E ? rows : (long long)E) + rows / kTileN) * ((a.N + chan - 1) / chan);
    const int grid = 2 * (int)(most < p.num_sms / 2 ? most : p.num_sms / 2);
    return launch_pdl(expert_gemm_kernel<kFp8, kSwiglu>, grid, kThreads, smem, s, mw, mx, a);
}

}  // namespace

bool encode_map(CUtensorMap *m, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
                const cuuint64_t *strides, const cuuint32_t *box) {
    using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    // the driver's function, found through the runtime: the library links no driver stub
    static const EncodeFn encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                                            &q) == cudaSuccess &&
                           q == cudaDriverEntryPointSuccess;
        return found ? reinterpret_cast<EncodeFn>(f) : nullptr;
    }();
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    // Rows that start on 128-byte lines are fetched ahead in pairs of lines; rows that do not would bring lines
    // in that belong to no box (8,168 rows of K = 1416: 125 us with, 111-119 us without; K = 1408: 85 us, 87 us).
    const CUtensorMapL2promotion promotion =
        strides[0] % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    return encode && encode(m, type, rank, const_cast<void *>(base), dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_expert_gemm(const a2av_plan_s &p, const MatmulArgs &a, bool fp8, bool swiglu, cudaStream_t s) {
    if (fp8) return swiglu ? launch_gemm<true, true>(p, a, s) : launch_gemm<true, false>(p, a, s);
    return swiglu ? launch_gemm<false, true>(p, a, s) : launch_gemm<false, false>(p, a, s);
}

}  // namespace a2av
