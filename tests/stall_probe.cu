// stall_probe.cu -- test helper, not part of libmoe: two warps wait on an
// mbarrier that nobody arrives at, with the waits of csrc/tc.cuh and a limit of
// MOE_STALL_NS (set by the test's build), then go through `later` more waits.
// Every wait is bounded, so the kernel ends by itself.
#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "tc.cuh"

namespace {

// out[0], out[1]: time of the first wait of warps 0 and 1; out[2], out[3]: time
// of their later waits; out[4], out[5]: result of the first wait and of the
// later ones (any of them true); out[6]: the flag; out[7]: the result and out[8]
// the flag of a wait on a phase that is over.
__global__ void stall_kernel(int later, unsigned long long* out) {
    __shared__ uint64_t never, once;
    __shared__ int gave_up;
    if (threadIdx.x == 0) {
        moe::mbar_init(&never, 1);
        moe::mbar_init(&once, 1);
        gave_up = 0;
        moe::mbar_init_fence();
        moe::mbar_arrive(&once);
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const bool ok = moe::mbar_wait(&once, 0, &gave_up);
        if (lane == 0) {
            out[7] = ok;
            out[8] = *(volatile int*)&gave_up;
        }
    }
    __syncthreads();
    const uint64_t t0 = moe::now_ns();
    bool first = false, any = false;
    if (warp == 0)
        first = moe::mbar_wait(&never, 0, &gave_up);
    else
        moe::mbar_pass(moe::smem_u32(&never), 0, &gave_up);
    const uint64_t t1 = moe::now_ns();
    for (int i = 0; i < later; ++i) {
        any |= moe::mbar_wait(&never, 0, &gave_up);
        moe::mbar_pass(moe::smem_u32(&never), 0, &gave_up);
    }
    const uint64_t t2 = moe::now_ns();
    if (lane == 0) {
        out[warp] = t1 - t0;
        out[2 + warp] = t2 - t1;
        if (warp == 0) {
            out[4] = first;
            out[5] = any;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) out[6] = gave_up;
}

}  // namespace

extern "C" __attribute__((visibility("default"))) int stall_run(int later, unsigned long long* out, void* stream) {
    stall_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(later, out);
    return (int)cudaGetLastError();
}
extern "C" __attribute__((visibility("default"))) long long stall_polls() { return moe::kStallPolls; }
extern "C" __attribute__((visibility("default"))) long long stall_poll_ns() { return moe::kPollNs; }
