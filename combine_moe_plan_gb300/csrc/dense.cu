// dense.cu -- the bf16 experts' grouped products and their gradients, for
// training: every expert's window of rows times its weights, forward and back.
//
//   up         g, u = x w13^T; h = silu(g) u; g and u kept as E4M3 codes
//   down       out = h w2^T
//   down_back  d = dout w2; back through the gates and the activation at the codes' values
//   up_back    dx = dgu w13
//   grad       dw = a^T b over the rows of a window
//
// Simple form: a CTA computes 32 rows by 256 columns, a column a thread, sums in
// fp32 registers, and finishes them from shared memory.
#include "moe_internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace moe {
namespace {

constexpr int kMostExperts = 4096;
constexpr int kTileM = 32, kTileN = 256;

enum class Op { kUp, kDown, kDownBack, kUpBack, kGrad };

struct Problem {
    int P, N, K;  // experts, outputs a row, inner size (of one half for up)
    const uint16_t* a;
    const uint16_t* w;
    const int32_t* offsets;
    int rows;
    uint16_t* out;      // up: h; down, up_back: the rows; down_back: hg
    uint16_t* dgu;      // down_back
    uint8_t* codes;     // up: out; down_back: in
    float* scales;
    int scale_stride;
    const float* row_gates;
    float* parts;
    void* dw;
    int grad;
    int32_t* err;
};

// Window p, if it lies inside the rows, runs forward and begins after every
// earlier offset; otherwise empty and reported.
__device__ __forceinline__ int2 window(const Problem& pr, int p) {
    const int lo = pr.offsets[p], hi = pr.offsets[p + 1];
    bool ok = lo >= 0 && hi >= lo && hi <= pr.rows;
    for (int q = 0; q < p; ++q) ok = ok && pr.offsets[q] <= lo;
    if (!ok && threadIdx.x == 0) set_error(pr.err, MOE_DEVERR_WINDOW);
    return ok ? make_int2(lo, hi) : make_int2(0, 0);
}

__device__ __forceinline__ float bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t to_bf16(float v) { return (uint16_t)(pack_bf16x2_rn(v, 0.0f) & 0xffffu); }
__device__ __forceinline__ float e4m3(uint8_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"((uint16_t)(h & 0xffffu)));
    return f;
}

template <Op OP>
__global__ void __launch_bounds__(kTileN) dense_kernel(const Problem pr) {
    __shared__ float a_tile[kTileM][33];
    __shared__ float y[kTileM][kTileN];
    grid_dependency_sync();
    allow_dependents();
    constexpr int kCols = OP == Op::kUp ? 128 : kTileN;  // outputs a tile
    const int p = blockIdx.y, n0 = blockIdx.x * kCols, c = threadIdx.x;
    const int2 win = window(pr, p);
    const int half = c >> 7;  // up: 0 gate, 1 up
    const int col = OP == Op::kUp ? n0 + (c & 127) : n0 + c;
    const bool col_ok = col < pr.N;
    const int groups = pr.N / 128;
    // grad: the tile's rows are columns of a, and the window's rows the inner dimension
    const int first = OP == Op::kGrad ? (int)blockIdx.z * kTileM : win.x;
    const int last = OP == Op::kGrad ? first + kTileM : win.y;
    const int K = OP == Op::kGrad ? win.y - win.x : pr.K;
    const int M = pr.K;  // grad: columns of a
    for (int m0 = first; m0 < last; m0 += kTileM) {
        float acc[kTileM];
#pragma unroll
        for (int r = 0; r < kTileM; ++r) acc[r] = 0.0f;
        for (int k0 = 0; k0 < K; k0 += 32) {
            __syncthreads();
            for (int i = c; i < kTileM * 32; i += kTileN) {
                float v = 0.0f;
                if (OP == Op::kGrad) {
                    const int kk = i / 32, r = i % 32;
                    if (k0 + kk < K) v = bf16(pr.a[(size_t)(win.x + k0 + kk) * M + m0 + r]);
                    a_tile[r][kk] = v;
                } else {
                    const int r = i / 32, kk = i % 32;
                    if (m0 + r < last) v = bf16(pr.a[(size_t)(m0 + r) * K + k0 + kk]);
                    a_tile[r][kk] = v;
                }
            }
            __syncthreads();
            for (int kk = 0; kk < 32 && k0 + kk < K; ++kk) {
                const int k = k0 + kk;
                float b = 0.0f;
                if (col_ok) {
                    if (OP == Op::kUp)
                        b = bf16(pr.w[((size_t)p * 2 * pr.N + half * pr.N + col) * K + k]);
                    else if (OP == Op::kDown)
                        b = bf16(pr.w[((size_t)p * pr.N + col) * K + k]);
                    else if (OP == Op::kGrad)
                        b = bf16(pr.w[(size_t)(win.x + k) * pr.N + col]);
                    else
                        b = bf16(pr.w[((size_t)p * K + k) * pr.N + col]);
                }
#pragma unroll
                for (int r = 0; r < kTileM; ++r) acc[r] = fmaf(a_tile[r][kk], b, acc[r]);
            }
        }
        if (OP == Op::kGrad) {
            if (!col_ok || (K == 0 && pr.grad == MOE_GRAD_F32_ADD)) continue;
#pragma unroll
            for (int r = 0; r < kTileM; ++r) {
                const size_t at = ((size_t)p * M + m0 + r) * pr.N + col;
                if (pr.grad == MOE_GRAD_BF16)
                    static_cast<uint16_t*>(pr.dw)[at] = to_bf16(acc[r]);
                else
                    static_cast<float*>(pr.dw)[at] = acc[r] + (pr.grad == MOE_GRAD_F32_ADD ? static_cast<float*>(pr.dw)[at] : 0.0f);
            }
            continue;
        }
#pragma unroll
        for (int r = 0; r < kTileM; ++r) y[r][c] = acc[r];
        __syncthreads();
        for (int r = 0; r < kTileM && m0 + r < last; ++r) {
            const size_t row = m0 + r;
            if (OP == Op::kDown || OP == Op::kUpBack) {
                if (col_ok) pr.out[row * pr.N + col] = to_bf16(y[r][c]);
            } else if (OP == Op::kUp) {
                if (half == 0) {
                    const float g = y[r][c], u = y[r][c + 128];
                    pr.out[row * pr.N + col] = to_bf16(g / (1.0f + expf(-g)) * u);
                }
                if (pr.codes != nullptr) {
                    float amax = 0.0f;
                    for (int i = 0; i < 128; ++i) amax = fmaxf(amax, fabsf(y[r][half * 128 + i]));
                    const float lift = amax < 0x1p-100f ? 0x1p64f : 1.0f;
                    const float inv = amax > 0.0f ? kE4M3Max / (amax * lift) : 0.0f;
                    pr.codes[row * 2 * pr.N + half * pr.N + col] = (uint8_t)(pack_e4m3x2(y[r][c] * lift * inv, 0.0f) & 0xff);
                    if ((c & 127) == 0) pr.scales[row * pr.scale_stride + half * groups + blockIdx.x] = amax / kE4M3Max;
                }
            } else if (col_ok) {
                const float* sc = pr.scales + row * pr.scale_stride + col / 128;
                const float g = e4m3(pr.codes[row * 2 * pr.N + col]) * sc[0];
                const float u = e4m3(pr.codes[row * 2 * pr.N + pr.N + col]) * sc[groups];
                const float s = 1.0f / (1.0f + expf(-g)), h = g * s * u, gate = pr.row_gates[row];
                const float d = y[r][c], dh = gate * d;
                pr.out[row * pr.N + col] = to_bf16(gate * h);
                pr.dgu[row * 2 * pr.N + col] = to_bf16(dh * u * s * (1.0f + g * (1.0f - s)));
                pr.dgu[row * 2 * pr.N + pr.N + col] = to_bf16(dh * g * s);
                y[r][c] = d * h;
            }
        }
        if (OP == Op::kDownBack) {
            __syncthreads();
            for (int i = c; i < kTileM * 2; i += kTileN) {
                const int r = i >> 1, b = i & 1;
                if (m0 + r < last && n0 + b * 128 < pr.N) {
                    float sum = 0.0f;
                    for (int j = 0; j < 128; ++j) sum += y[r][b * 128 + j];
                    pr.parts[(size_t)(m0 + r) * groups + n0 / 128 + b] = sum;
                }
            }
        }
    }
}

template <Op OP>
int launch_dense(const Problem& pr, int m_tiles, cudaStream_t s) {
    constexpr int kCols = OP == Op::kUp ? 128 : kTileN;
    const dim3 grid((unsigned)((pr.N + kCols - 1) / kCols), (unsigned)pr.P, (unsigned)m_tiles);
    return launch_pdl(dense_kernel<OP>, grid, dim3(kTileN), 0, s, pr) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dense(const moe_dense* e, int32_t rows) {
    if (e == nullptr || e->error_word == nullptr) return MOE_ERR_NULL;
    if (e->P < 1 || e->P > kMostExperts) return MOE_ERR_SIZE;
    if (e->H < kGroup || e->H > 65536 || e->H % kGroup != 0) return MOE_ERR_SIZE;
    if (e->I < kGroup || e->I > 65536 || e->I % kGroup != 0) return MOE_ERR_SIZE;
    if (rows < 0 || rows > INT32_MAX / 2) return MOE_ERR_SIZE;
    return aligned16(e->error_word) ? MOE_OK : MOE_ERR_ALIGN;
}

// Pointers that a call over `rows` rows needs.
template <size_t N>
int check_pointers(const void* const (&need)[N], int32_t rows) {
    for (const void* p : need) {
        if (rows > 0 && p == nullptr) return MOE_ERR_NULL;
        if (!aligned16(p)) return MOE_ERR_ALIGN;
    }
    return MOE_OK;
}

bool stride_ok(int32_t stride, int32_t width) { return stride % 4 == 0 && stride >= width / kGroup; }

// The gradient of weights [P, M, N] from a [rows, M] and b [rows, N].
int grad_call(const moe_dense* e, int M, int N, const uint16_t* a, const uint16_t* b, const int32_t* offsets,
              int32_t rows, void* dw, int32_t grad, cudaStream_t s) {
    int rc = check_dense(e, rows);
    if (rc != MOE_OK) return rc;
    if (grad < MOE_GRAD_F32 || grad > MOE_GRAD_BF16) return MOE_ERR_SIZE;
    if (dw == nullptr) return MOE_ERR_NULL;
    if (!aligned16(dw)) return MOE_ERR_ALIGN;
    const void* need[] = {a, b, offsets};
    if ((rc = check_pointers(need, rows)) != MOE_OK) return rc;
    if (rows == 0) {
        if (grad == MOE_GRAD_F32_ADD) return MOE_OK;
        const size_t bytes = (size_t)e->P * M * N * (grad == MOE_GRAD_BF16 ? 2 : 4);
        return cudaMemsetAsync(dw, 0, bytes, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    Problem pr = {};
    pr.P = e->P, pr.N = N, pr.K = M, pr.a = a, pr.w = b, pr.offsets = offsets, pr.rows = rows;
    pr.dw = dw, pr.grad = grad, pr.err = e->error_word;
    return launch_dense<Op::kGrad>(pr, M / kTileM, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_dense_up(const moe_dense* e, const uint16_t* x, const int32_t* offsets, int32_t rows,
                                    uint16_t* h, uint8_t* codes, float* scales, int32_t scale_stride, void* stream) {
    int rc = check_dense(e, rows);
    if (rc != MOE_OK) return rc;
    const bool keep = codes != nullptr || scales != nullptr;
    if (keep && !stride_ok(scale_stride, 2 * e->I)) return MOE_ERR_SIZE;
    const void* need[] = {e->w13, x, offsets, h, keep ? codes : static_cast<const void*>(h),
                          keep ? scales : static_cast<const void*>(h)};
    if ((rc = check_pointers(need, rows)) != MOE_OK || rows == 0) return rc;
    Problem pr = {};
    pr.P = e->P, pr.N = e->I, pr.K = e->H, pr.a = x, pr.w = e->w13, pr.offsets = offsets, pr.rows = rows, pr.out = h;
    pr.codes = codes, pr.scales = scales, pr.scale_stride = scale_stride, pr.err = e->error_word;
    return launch_dense<Op::kUp>(pr, 1, static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API int moe_dense_down(const moe_dense* e, const uint16_t* h, const int32_t* offsets, int32_t rows,
                                      uint16_t* out, void* stream) {
    int rc = check_dense(e, rows);
    if (rc != MOE_OK) return rc;
    const void* need[] = {e->w2, h, offsets, out};
    if ((rc = check_pointers(need, rows)) != MOE_OK || rows == 0) return rc;
    Problem pr = {};
    pr.P = e->P, pr.N = e->H, pr.K = e->I, pr.a = h, pr.w = e->w2, pr.offsets = offsets, pr.rows = rows, pr.out = out;
    pr.err = e->error_word;
    return launch_dense<Op::kDown>(pr, 1, static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API int moe_dense_down_backward(const moe_dense* e, const uint16_t* dout, const uint8_t* codes,
                                               const float* scales, int32_t scale_stride, const float* row_gates,
                                               const int32_t* offsets, int32_t rows, uint16_t* dgu, uint16_t* hg,
                                               float* gate_parts, void* stream) {
    int rc = check_dense(e, rows);
    if (rc != MOE_OK) return rc;
    if (!stride_ok(scale_stride, 2 * e->I)) return MOE_ERR_SIZE;
    const void* need[] = {e->w2, dout, codes, scales, row_gates, offsets, dgu, hg, gate_parts};
    if ((rc = check_pointers(need, rows)) != MOE_OK || rows == 0) return rc;
    Problem pr = {};
    pr.P = e->P, pr.N = e->I, pr.K = e->H, pr.a = dout, pr.w = e->w2, pr.offsets = offsets, pr.rows = rows;
    pr.out = hg, pr.dgu = dgu, pr.codes = const_cast<uint8_t*>(codes), pr.scales = const_cast<float*>(scales);
    pr.scale_stride = scale_stride, pr.row_gates = row_gates, pr.parts = gate_parts, pr.err = e->error_word;
    return launch_dense<Op::kDownBack>(pr, 1, static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API int moe_dense_up_backward(const moe_dense* e, const uint16_t* dgu, const int32_t* offsets,
                                             int32_t rows, uint16_t* dx, void* stream) {
    int rc = check_dense(e, rows);
    if (rc != MOE_OK) return rc;
    const void* need[] = {e->w13, dgu, offsets, dx};
    if ((rc = check_pointers(need, rows)) != MOE_OK || rows == 0) return rc;
    Problem pr = {};
    pr.P = e->P, pr.N = e->H, pr.K = 2 * e->I, pr.a = dgu, pr.w = e->w13, pr.offsets = offsets, pr.rows = rows;
    pr.out = dx, pr.err = e->error_word;
    return launch_dense<Op::kUpBack>(pr, 1, static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API int moe_dense_up_grad(const moe_dense* e, const uint16_t* dgu, const uint16_t* x,
                                         const int32_t* offsets, int32_t rows, void* dw13, int32_t grad, void* stream) {
    return grad_call(e, e == nullptr ? 0 : 2 * e->I, e == nullptr ? 0 : e->H, dgu, x, offsets, rows, dw13, grad,
                     static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API int moe_dense_down_grad(const moe_dense* e, const uint16_t* dout, const uint16_t* hg,
                                           const int32_t* offsets, int32_t rows, void* dw2, int32_t grad,
                                           void* stream) {
    return grad_call(e, e == nullptr ? 0 : e->H, e == nullptr ? 0 : e->I, dout, hg, offsets, rows, dw2, grad,
                     static_cast<cudaStream_t>(stream));
}
