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
// token's copies (and, for softmax scores, over its logits).  Renormalised scores are
// divided by their sum S before anything else: r_j = s_j / S is at most 1, where
// (dg_j - sum_i dg_i r_i) / S overflows once all scores of a token are tiny, although
// its product with s_j is of dg's size.
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

// KEEP: logits a lane holds (softmax scores; at least E / 32).  QUADS: the partial
// sums are read 16 bytes at a time (their number a multiple of 4).
template <Gates KIND, int KEEP, bool QUADS>
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
    const bool chosen = lane < k;
    const int my_slot = chosen ? slot[copy] : 0, my_e = chosen ? topk_e[copy] : 0;
    const float* row = logits + (size_t)t * E;
    float l[KEEP];
    if constexpr (KIND == Gates::kSoftmax) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) l[i] = lane + 32 * i < E ? row[lane + 32 * i] : -INFINITY;
    }
    const float gate = KIND == Gates::kPlan && chosen ? gates[copy] : 0.0f;
    if (__any_sync(kFull, my_slot < 0 || my_slot >= T * k || my_e < 0 || my_e >= E)) {
        if (lane == 0) set_error(err, MOE_DEVERR_SLOT);
        return;
    }
    const float mine = KIND != Gates::kPlan && chosen ? row[my_e] : 0.0f;

    // dg of copy `lane`: `lanes` lanes a copy, 32 / lanes copies at a time
    const int in_run = lane & (lanes - 1), run = lane / lanes, runs = 32 / lanes;
    float dg = 0.0f;
    for (int j0 = 0; j0 < k; j0 += runs) {
        const int j = j0 + run;
        const float* p = gate_parts + (size_t)__shfl_sync(kFull, my_slot, j & 31) * parts;
        float sum = 0.0f;
        if (j < k) {
            if (QUADS) {
                for (int b = in_run * 4; b < parts; b += lanes * 4) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(p + b));
                    sum += (v.x + v.y) + (v.z + v.w);
                }
            } else {
                for (int b = in_run; b < parts; b += lanes) sum += p[b];
            }
        }
        for (int off = lanes >> 1; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
        // run r holds copy j0 + r: to lane j0 + r
        const float v = __shfl_sync(kFull, sum, ((lane - j0) & (runs - 1)) * lanes);
        if (lane >= j0 && lane < j0 + runs) dg = v;
    }
    if (chosen)
        dgates[copy] = dg;
    else
        dg = 0.0f;

    float* out = dlogits + (size_t)t * E;
    if constexpr (KIND == Gates::kPlan) {
        const float mean = warp_sum(gate * dg);
        for (int e = lane; e < E; e += 32) out[e] = 0.0f;
        __syncwarp();
        if (chosen) out[my_e] = gate * (dg - mean);
        return;
    }
    float top = -INFINITY, total = 0.0f;
    if constexpr (KIND == Gates::kSoftmax) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) top = fmaxf(top, l[i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            l[i] = finite_or_zero(expf(l[i] - top));
            total += l[i];
        }
        total = warp_sum(total);
    }
    const float s = !chosen                    ? 0.0f
                    : KIND == Gates::kSigmoid  ? finite_or_zero(1.0f / (1.0f + expf(-mine)))
                                               : finite_or_zero(expf(mine - top) / total);
    // ds_j s_j of a chosen copy
    float dss = scale * dg * s;
    if (renorm) {
        const float sum = warp_sum(s);
        const float r = sum > 0.0f ? s / sum : 0.0f;
        dss = scale * (dg - warp_sum(dg * r)) * r;
    }
    if (KIND == Gates::kSigmoid || renorm) {  // (the sum of dss is 0 with renorm, so that the others have no part in a softmax)
        for (int e = lane; e < E; e += 32) out[e] = 0.0f;
        __syncwarp();
        if (chosen) out[my_e] = KIND == Gates::kSigmoid ? dss * (1.0f - s) : dss;
    } else {
        const float mean = warp_sum(dss);
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (lane + 32 * i < E) out[lane + 32 * i] = -finite_or_zero(l[i] / total) * mean;
        __syncwarp();
        if (chosen) out[my_e] = dss - s * mean;
    }
}

using GatesKernel = decltype(&gates_backward_kernel<Gates::kPlan, 1, false>);

template <bool QUADS>
GatesKernel gates_kernel(const moe_router* router, int E) {
    if (router == nullptr) return gates_backward_kernel<Gates::kPlan, 1, QUADS>;
    if (router->score == MOE_SCORE_SIGMOID) return gates_backward_kernel<Gates::kSigmoid, 1, QUADS>;
    return E <= 64    ? gates_backward_kernel<Gates::kSoftmax, 2, QUADS>
           : E <= 256 ? gates_backward_kernel<Gates::kSoftmax, 8, QUADS>
                      : gates_backward_kernel<Gates::kSoftmax, 32, QUADS>;
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
    const bool quads = parts % 4 == 0;
    const int loads = quads ? parts / 4 : parts;
    int lanes = 1;
    while (lanes < 32 && lanes < loads) lanes *= 2;
    const GatesKernel kernel = quads ? gates_kernel<true>(router, E) : gates_kernel<false>(router, E);
    const bool renorm = router != nullptr && router->renorm != 0;
    const float scale = router != nullptr ? router->scale : 1.0f;
    const int blocks = (T + kGatesThreads / 32 - 1) / (kGatesThreads / 32);
    const cudaError_t e = launch_pdl(kernel, dim3((unsigned)blocks), dim3(kGatesThreads), 0, s, logits, gates, topk_e,
                                     slot, gate_parts, parts, T, E, k, renorm, scale, lanes, dgates, dlogits, err);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace moe
