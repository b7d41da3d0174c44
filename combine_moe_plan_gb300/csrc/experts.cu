// experts.cu -- the experts' grouped products on E4M3 rows and weights.
//
//   y[r, n] = sum_b sa[r, b] sw[n / 128, b] sum_{i in block b} a[r, i] w[n, i]
//
// for every row r of expert p's window and every output n, with b the
// 128-element blocks of the inner dimension.  moe_experts_up computes gate and
// up outputs of the same 128 columns, h = silu(gate) up, and quantizes the 128
// values of each row as one group; moe_experts_down rounds y to bf16.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int kRowTile = 16;  // rows a CTA accumulates at a time

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

// One CTA per (128 output columns, expert); a thread owns one column (UP: the
// gate and the up column) of kRowTile rows at a time.
template <bool UP>
__global__ void __launch_bounds__(kGroup)
experts_kernel(int P, int N, int K, const uint8_t* __restrict__ a, const float* __restrict__ sa, int sa_stride,
               const uint8_t* __restrict__ w, const float* __restrict__ sw, const int32_t* __restrict__ offsets,
               int rows, uint8_t* __restrict__ h, float* __restrict__ hs, int hs_stride, uint16_t* __restrict__ out,
               int32_t* __restrict__ err) {
    __shared__ float s_a[kRowTile][kGroup];
    __shared__ float s_max[kGroup / 32][kRowTile];
    grid_dependency_sync();
    allow_dependents();
    const int p = blockIdx.y, nb = blockIdx.x, c = threadIdx.x;
    const int lo = offsets[p], hi = offsets[p + 1];
    if (lo < 0 || hi < lo || hi > rows) {
        if (c == 0) set_error(err, MOE_DEVERR_WINDOW);
        return;
    }
    const int kb = K / kGroup, width = UP ? 2 * N : N;  // N: output columns
    const int n = nb * kGroup + c;
    const uint8_t* w0 = w + ((size_t)p * width + n) * K;
    const uint8_t* w1 = w0 + (size_t)N * K;
    const float* sw0 = sw + ((size_t)p * (width / kGroup) + nb) * kb;
    const float* sw1 = sw0 + (size_t)(N / kGroup) * kb;
    for (int r0 = lo; r0 < hi; r0 += kRowTile) {
        const int nr = min(kRowTile, hi - r0);
        float y0[kRowTile], y1[kRowTile];
#pragma unroll
        for (int r = 0; r < kRowTile; ++r) y0[r] = y1[r] = 0.0f;
        for (int b = 0; b < kb; ++b) {
            __syncthreads();
            for (int r = 0; r < kRowTile; ++r)
                s_a[r][c] = r < nr ? e4m3_value(a[(size_t)(r0 + r) * K + b * kGroup + c]) : 0.0f;
            __syncthreads();
            float t0[kRowTile], t1[kRowTile];
#pragma unroll
            for (int r = 0; r < kRowTile; ++r) t0[r] = t1[r] = 0.0f;
            for (int i = 0; i < kGroup; ++i) {
                const float v0 = e4m3_value(w0[b * kGroup + i]);
                const float v1 = UP ? e4m3_value(w1[b * kGroup + i]) : 0.0f;
#pragma unroll
                for (int r = 0; r < kRowTile; ++r) {
                    t0[r] = fmaf(s_a[r][i], v0, t0[r]);
                    if (UP) t1[r] = fmaf(s_a[r][i], v1, t1[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < kRowTile; ++r) {
                if (r < nr) {
                    const float f = sa[(size_t)(r0 + r) * sa_stride + b];
                    y0[r] = fmaf(f * sw0[b], t0[r], y0[r]);
                    if (UP) y1[r] = fmaf(f * sw1[b], t1[r], y1[r]);
                }
            }
        }
        if (!UP) {
            for (int r = 0; r < nr; ++r)
                out[(size_t)(r0 + r) * N + n] = (uint16_t)(pack_bf16x2_rn(y0[r], 0.0f) & 0xffffu);
            continue;
        }
#pragma unroll
        for (int r = 0; r < kRowTile; ++r) {
            y0[r] = y0[r] / (1.0f + expf(-y0[r])) * y1[r];
            const unsigned m = __reduce_max_sync(kFull, __float_as_uint(fabsf(y0[r])));
            if ((c & 31) == 0) s_max[c / 32][r] = __uint_as_float(m);
        }
        __syncthreads();
        for (int r = 0; r < nr; ++r) {
            const float m = fmaxf(fmaxf(s_max[0][r], s_max[1][r]), fmaxf(s_max[2][r], s_max[3][r]));
            const float den = m > 0.0f ? m : 1.0f;
            h[(size_t)(r0 + r) * N + n] = (uint8_t)(pack_e4m3x2(y0[r] * kE4M3Max / den, 0.0f) & 0xffu);
            if (c == 0) hs[(size_t)(r0 + r) * hs_stride + nb] = m / kE4M3Max;
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_experts(const moe_experts* e) {
    if (e == nullptr || e->error_word == nullptr) return MOE_ERR_NULL;
    if (e->P < 1 || e->P > 4096) return MOE_ERR_SIZE;
    if (e->H < kGroup || e->H > 65536 || e->H % kGroup != 0) return MOE_ERR_SIZE;
    if (e->I < kGroup || e->I > 65536 || e->I % kGroup != 0) return MOE_ERR_SIZE;
    if (!aligned16(e->error_word)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

bool stride_ok(int32_t stride, int32_t width) { return stride % 4 == 0 && stride >= width / kGroup; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_experts_up(const moe_experts* e, const uint8_t* codes, const float* scales,
                                      int32_t scale_stride, const int32_t* offsets, int32_t rows, uint8_t* h,
                                      float* h_scales, int32_t h_stride, void* stream) {
    int rc = check_experts(e);
    if (rc != MOE_OK) return rc;
    if (rows < 0 || rows > INT32_MAX / 2) return MOE_ERR_SIZE;
    if (!stride_ok(scale_stride, e->H) || !stride_ok(h_stride, e->I)) return MOE_ERR_SIZE;
    const void* need[] = {e->w13, e->s13, codes, scales, offsets, h, h_scales};
    for (const void* p : need) {
        if (rows > 0 && p == nullptr) return MOE_ERR_NULL;
        if (!aligned16(p)) return MOE_ERR_ALIGN;
    }
    if (rows == 0) return MOE_OK;
    cudaError_t c = launch_pdl(experts_kernel<true>, dim3(e->I / kGroup, e->P), dim3(kGroup), 0,
                               static_cast<cudaStream_t>(stream), e->P, e->I, e->H, codes, scales, scale_stride,
                               e->w13, e->s13, offsets, rows, h, h_scales, h_stride, (uint16_t*)nullptr,
                               e->error_word);
    return c == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API int moe_experts_down(const moe_experts* e, const uint8_t* h, const float* h_scales,
                                        int32_t h_stride, const int32_t* offsets, int32_t rows, uint16_t* out,
                                        void* stream) {
    int rc = check_experts(e);
    if (rc != MOE_OK) return rc;
    if (rows < 0 || rows > INT32_MAX / 2) return MOE_ERR_SIZE;
    if (!stride_ok(h_stride, e->I)) return MOE_ERR_SIZE;
    const void* need[] = {e->w2, e->s2, h, h_scales, offsets, out};
    for (const void* p : need) {
        if (rows > 0 && p == nullptr) return MOE_ERR_NULL;
        if (!aligned16(p)) return MOE_ERR_ALIGN;
    }
    if (rows == 0) return MOE_OK;
    cudaError_t c = launch_pdl(experts_kernel<false>, dim3(e->H / kGroup, e->P), dim3(kGroup), 0,
                               static_cast<cudaStream_t>(stream), e->P, e->H, e->I, h, h_scales, h_stride, e->w2,
                               e->s2, offsets, rows, (uint8_t*)nullptr, (float*)nullptr, 0, out, e->error_word);
    return c == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
