// plan_routed.cu -- moe_plan_routed's kernels: the plan (plan_kernels.cuh) with
// a scored router (sigmoid or softmax scores, balance bias, expert groups).
#include "plan_kernels.cuh"

namespace moe {

cudaError_t launch_plan_routed(const moe_router& r, const float* bias, const float* logits, int T, int E, int P,
                               int k, const int32_t* rep_off, const int32_t* rep_ids, int32_t* topk_e, float* gates,
                               int32_t* phys, int32_t* tile_hist, int32_t* local_rank, int32_t* counts,
                               int32_t* offsets, int32_t* slot, int32_t* src_token, int32_t* src_k, int32_t* err,
                               int32_t* ticket, cudaStream_t s, uint64_t* launches) {
    const ScoreRouter router = {bias,         r.scale, r.score == MOE_SCORE_SIGMOID, r.n_group,
                                r.topk_group, r.group_top, r.renorm != 0};
    return launch_plan_with(router, logits, T, E, P, k, rep_off, rep_ids, topk_e, gates, phys, tile_hist, local_rank,
                            counts, offsets, slot, src_token, src_k, err, ticket, s, launches);
}

}  // namespace moe
