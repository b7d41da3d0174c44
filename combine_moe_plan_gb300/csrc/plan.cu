// plan.cu -- moe_plan's kernels: the plan (plan_kernels.cuh) with the
// framework's own router, a softmax over the k largest logits.
#include "plan_kernels.cuh"

namespace moe {

#ifdef MOE_TRACE
int trace_symbols_plan(int kind, void** stamps, void** sms) {
    cudaError_t e = cudaErrorInvalidValue;
    switch (kind) {
        case kTraceRoute:
            e = cudaGetSymbolAddress(stamps, tr_route_t);
            if (e == cudaSuccess) e = cudaGetSymbolAddress(sms, tr_route_sm);
            break;
        case kTraceColumnScan:
            e = cudaGetSymbolAddress(stamps, tr_scan_t);
            if (e == cudaSuccess) e = cudaGetSymbolAddress(sms, tr_scan_sm);
            break;
        case kTraceAssign:
            e = cudaGetSymbolAddress(stamps, tr_assign_t);
            if (e == cudaSuccess) e = cudaGetSymbolAddress(sms, tr_assign_sm);
            break;
        case kTracePlanSingle:
            e = cudaGetSymbolAddress(stamps, tr_single_t);
            if (e == cudaSuccess) e = cudaGetSymbolAddress(sms, tr_single_sm);
            break;

        default:
            break;
    }
    return e == cudaSuccess ? 0 : -1;
}
#endif

cudaError_t launch_plan(const float* logits, int T, int E, int P, int k, const int32_t* rep_off,
                        const int32_t* rep_ids, int32_t* topk_e, float* gates, int32_t* phys,
                        int32_t* tile_hist, int32_t* local_rank, int32_t* counts, int32_t* offsets,
                        int32_t* slot, int32_t* src_token, int32_t* src_k, int32_t* err, int32_t* ticket,
                        cudaStream_t s, uint64_t* launches) {
    return launch_plan_with(TopkSoftmax{}, logits, T, E, P, k, rep_off, rep_ids, topk_e, gates, phys, tile_hist,
                            local_rank, counts, offsets, slot, src_token, src_k, err, ticket, s, launches);
}

}  // namespace moe
