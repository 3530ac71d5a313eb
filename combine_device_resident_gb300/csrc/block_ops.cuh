// Arguments and launchers of the router by scores, the gradients of router and
// combine, and the norms around a block.
#pragma once
#include "a2av_internal.cuh"

namespace a2av {

constexpr int kMaxGroups = 64;          // expert groups: two per lane
constexpr int kMaxNormGradRow = 16384;  // row length of the norms' gradient: its weights' sums lie in shared memory

struct ScoreArgs {
    Geometry g;
    const int32_t *num_tokens;
    const float *logits, *bias;  // bias may be null
    int32_t *idx;                // out, or (gradient) in
    float *gate;                 // out
    const float *d_gate;         // gradient
    float *d_logits;
    uint32_t *status;
    int32_t sigmoid, groups, kept, best, renorm;
    float scale;
};

struct CombineGradArgs {
    Geometry g;
    const int32_t *num_tokens;
    const uint16_t *d_out, *y;  // y null without d_gate
    const float *gate;          // null without d_y
    const int32_t *slot_map;
    uint16_t *d_y;  // may be null
    float *d_gate;  // may be null
    int64_t arena_rows;
    uint32_t *status;
};

struct BlockNormArgs {
    Geometry g;
    const int32_t *num_tokens;
    const uint16_t *x, *residual;
    const uint16_t *post, *gate, *weight;  // may be null
    int32_t gate_kind;
    float residual_scale, branch_scale, eps;
    uint16_t *residual_out, *y;  // may be null
    uint8_t *rows8;              // may be null
    // gradient
    const uint16_t *d_y, *d_residual_out;  // may be null
    uint16_t *d_x, *d_residual;
    float *d_weight, *d_post;  // may be null
    void *d_gate;              // may be null
    float *scratch;            // [blocks][2][H]: a block's sums for the weight, and for post_weight and gate together
};

cudaError_t launch_route_scores(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s);
cudaError_t launch_route_scores_grad(const a2av_plan_s &p, const ScoreArgs &a, cudaStream_t s);
cudaError_t launch_combine_grad(const a2av_plan_s &p, const CombineGradArgs &a, cudaStream_t s);
cudaError_t launch_block_norm(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s);
// `launches` is raised by the kernels enqueued.
cudaError_t launch_block_norm_grad(const a2av_plan_s &p, const BlockNormArgs &a, cudaStream_t s, int64_t &launches);
int64_t norm_scratch_bytes(const a2av_plan_s &p);

}  // namespace a2av
