// rows.cu -- the token side of training: bf16 rows into the expert windows, and
// the gradients of the gates and the router's logits.
//
// scatter_kernel: rows[slot[t, j]] = x[t].  One warp per (token, 512 elements):
// a lane holds two 16-byte chunks and writes them k times; x is read once.  Bound
// by HBM writes.
//
// gates_backward_kernel: one warp per token.  A copy's partial sums are added by a
// power-of-two run of lanes, several copies side by side, always in the same
// order; lane j then holds dg_j, and the router's gradient needs two sums over the
// token's copies (and, for softmax scores, over its logits).
#include "moe_internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kScatterThreads = 256;
constexpr int kScatterSeg = 512;  // elements per warp: two 16-byte chunks a lane

__global__ void __launch_bounds__(kScatterThreads)
scatter_kernel(const uint16_t* __restrict__ x, int T, int H, int k, const int32_t* __restrict__ slot,
               const float* __restrict__ gates, uint16_t* __restrict__ rows, float* __restrict__ row_gates,
               int32_t* __restrict__ err) {
    grid_dependency_sync();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int segs = (H + kScatterSeg - 1) / kScatterSeg;
    const long long item = (long long)blockIdx.x * (kScatterThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(item / segs);
    const int seg = (int)(item - (long long)t * segs);
    if (t >= T) return;

    const int c0 = seg * kScatterSeg + lane * 8, c1 = c0 + kScatterSeg / 2;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (c0 < H) a = ld_stream16(x + (size_t)t * H + c0);
    if (c1 < H) b = ld_stream16(x + (size_t)t * H + c1);
    const int my_slot = lane < k ? slot[(size_t)t * k + lane] : 0;
    if (__any_sync(kFull, my_slot < 0 || my_slot >= T * k)) {
        if (lane == 0) set_error(err, MOE_DEVERR_SLOT);
        return;
    }
    if (seg == 0 && row_gates != nullptr && lane < k) row_gates[my_slot] = gates[(size_t)t * k + lane];
    for (int j = 0; j < k; ++j) {
        uint16_t* dst = rows + (size_t)__shfl_sync(kFull, my_slot, j) * H;
        if (c0 < H) st16(dst + c0, a);
        if (c1 < H) st16(dst + c1, b);
    }
}

constexpr int kGatesThreads = 256;

enum class Gates { kPlan, kSigmoid, kSoftmax };

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}
__device__ __forceinline__ float finite_or_zero(float s) { return s == s ? s : 0.0f; }  // NaN counts as score 0

template <Gates KIND>
__global__ void __launch_bounds__(kGatesThreads)
gates_backward_kernel(const float* __restrict__ logits, const float* __restrict__ gates,
                      const int32_t* __restrict__ topk_e, const int32_t* __restrict__ slot,
                      const float* __restrict__ gate_parts, int parts, int T, int E, int k, bool renorm, float scale,
                      int lanes, float* __restrict__ dgates, float* __restrict__ dlogits, int32_t* __restrict__ err) {
    grid_dependency_sync();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kGatesThreads / 32) + (threadIdx.x >> 5);
    if (t >= T) return;
    const size_t copy = (size_t)t * k + lane;
    const int my_slot = lane < k ? slot[copy] : 0, my_e = lane < k ? topk_e[copy] : 0;
    if (__any_sync(kFull, my_slot < 0 || my_slot >= T * k || my_e < 0 || my_e >= E)) {
        if (lane == 0) set_error(err, MOE_DEVERR_SLOT);
        return;
    }

    // dg of copy `lane`: `lanes` lanes a copy, 32 / lanes copies at a time
    const int in_run = lane & (lanes - 1), run = lane / lanes, runs = 32 / lanes;
    float dg = 0.0f;
    for (int j0 = 0; j0 < k; j0 += runs) {
        const int j = j0 + run;
        const int s = __shfl_sync(kFull, my_slot, j & 31);
        float sum = 0.0f;
        if (j < k)
            for (int b = in_run; b < parts; b += lanes) sum += gate_parts[(size_t)s * parts + b];
        for (int off = lanes >> 1; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
        // run r holds copy j0 + r: to lane j0 + r
        const float mine = __shfl_sync(kFull, sum, ((lane - j0) & (runs - 1)) * lanes);
        if (lane >= j0 && lane < j0 + runs) dg = mine;
    }
    if (lane < k) dgates[copy] = dg;
    const bool chosen = lane < k;
    if (!chosen) dg = 0.0f;

    float* out = dlogits + (size_t)t * E;
    if constexpr (KIND == Gates::kPlan) {
        const float g = chosen ? gates[copy] : 0.0f;
        const float mean = warp_sum(g * dg);
        for (int e = lane; e < E; e += 32) out[e] = 0.0f;
        __syncwarp();
        if (chosen) out[my_e] = g * (dg - mean);
        return;
    }
    const float* row = logits + (size_t)t * E;
    float top = -INFINITY, total = 0.0f;
    if constexpr (KIND == Gates::kSoftmax) {
        for (int e = lane; e < E; e += 32) top = fmaxf(top, row[e]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        for (int e = lane; e < E; e += 32) total += finite_or_zero(expf(row[e] - top));
        total = warp_sum(total);
    }
    const auto score = [&](float l) {
        return finite_or_zero(KIND == Gates::kSigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / total);
    };
    const float s = chosen ? score(row[my_e]) : 0.0f;
    float ds = scale * dg;
    if (renorm) {
        const float sum = warp_sum(s);
        const float mean = warp_sum(ds * s) / sum;
        ds = chosen && sum > 0.0f ? (ds - mean) / sum : 0.0f;
    }
    if constexpr (KIND == Gates::kSigmoid) {
        for (int e = lane; e < E; e += 32) out[e] = 0.0f;
        __syncwarp();
        if (chosen) out[my_e] = ds * s * (1.0f - s);
    } else {
        const float mean = warp_sum(ds * s);
        for (int e = lane; e < E; e += 32) out[e] = -score(row[e]) * mean;
        __syncwarp();
        if (chosen) out[my_e] = s * (ds - mean);
    }
}

}  // namespace

cudaError_t launch_scatter(const uint16_t* x, int T, int H, int k, const int32_t* slot, const float* gates,
                           uint16_t* rows, float* row_gates, int32_t* err, cudaStream_t s, uint64_t* launches) {
    const long long items = (long long)T * ((H + kScatterSeg - 1) / kScatterSeg);
    const long long blocks = (items + kScatterThreads / 32 - 1) / (kScatterThreads / 32);
    const cudaError_t e = launch_pdl(scatter_kernel, dim3((unsigned)blocks), dim3(kScatterThreads), 0, s, x, T, H, k,
                                     slot, gates, rows, row_gates, err);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

cudaError_t launch_gates_backward(const moe_router* router, const float* logits, const float* gates,
                                  const int32_t* topk_e, const int32_t* slot, const float* gate_parts, int parts,
                                  int T, int E, int k, float* dgates, float* dlogits, int32_t* err, cudaStream_t s,
                                  uint64_t* launches) {
    int lanes = 1;
    while (lanes < 32 && lanes < parts) lanes *= 2;
    const auto kernel = router == nullptr                      ? gates_backward_kernel<Gates::kPlan>
                        : router->score == MOE_SCORE_SIGMOID   ? gates_backward_kernel<Gates::kSigmoid>
                                                               : gates_backward_kernel<Gates::kSoftmax>;
    const bool renorm = router != nullptr && router->renorm != 0;
    const float scale = router != nullptr ? router->scale : 1.0f;
    const int blocks = (T + kGatesThreads / 32 - 1) / (kGatesThreads / 32);
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)blocks), dim3(kGatesThreads), 0, s, logits, gates, topk_e,
                                     slot, gate_parts, parts, T, E, k, renorm, scale, lanes, dgates, dlogits, err);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace moe
