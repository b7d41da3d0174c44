// pair_probe.cu -- test helper, not part of libmoe: a cluster of two CTAs with the
// barriers of csrc/tc.cuh.  CTA 1 arrives at a barrier of CTA 0 in the ways that the
// bf16 products use, and CTA 0 waits for it; then both wait on a barrier that nobody
// arrives at, with a limit of MOE_STALL_NS (set by the test's build).  Every wait is
// bounded, so the kernel ends by itself.
#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "tc.cuh"

namespace {

// out[0]: whether CTA 0's waits for `rounds` phases, of two arrivals of CTA 1 each,
// and CTA 1's for one of CTA 0's between them, all ended; out[1]: the rounds;
// out[2 + rank]: whether the endless wait was left, out[4 + rank]: its time;
// out[6 + rank]: the longest of eight polls by themselves (how long a poll sleeps is
// the hardware's choice: the time it is given is a hint).
__global__ void __cluster_dims__(2, 1, 1) pair_kernel(int rounds, unsigned long long* out) {
    __shared__ uint64_t ready, taken, never;
    __shared__ int gave_up;
    const uint32_t rank = moe::cluster_ctarank();
    if (threadIdx.x == 0) {
        moe::mbar_init(&ready, 2);
        moe::mbar_init(&taken, 1);
        moe::mbar_init(&never, 1);
        moe::mbar_init_fence();
        gave_up = 0;
    }
    moe::cluster_arrive();
    moe::cluster_wait();
    if (threadIdx.x == 0) {
        const uint32_t there = moe::peer_smem(moe::smem_u32(&ready), 0), back = moe::peer_smem(moe::smem_u32(&taken), 1);
        bool ok = true;
        unsigned long long done = 0;
        for (int i = 0; ok && i < rounds; ++i) {
            if (rank == 1) {
                moe::mbar_signal_cluster(there);
                moe::mbar_arrive_cluster(there);
                ok = moe::mbar_wait_pair(&taken, i & 1, &gave_up);
            } else {
                ok = moe::mbar_wait_pair(&ready, i & 1, &gave_up);
                ++done;
                moe::mbar_arrive_cluster(back);
            }
        }
        if (rank == 0) {
            out[0] = ok;
            out[1] = done;
        }
        uint64_t longest = 0;
        for (int i = 0; i < 8; ++i) {
            const uint64_t t = moe::now_ns();
            if (moe::PairPhase{moe::smem_u32(&never), 0}.poll()) break;  // (waits for the answer; there is none)
            const uint64_t d = moe::now_ns() - t;
            longest = d > longest ? d : longest;
        }
        out[6 + rank] = longest;
        const uint64_t t0 = moe::now_ns();
        out[2 + rank] = !moe::mbar_wait_pair(&never, 0, &gave_up) && gave_up;
        out[4 + rank] = moe::now_ns() - t0;
    }
    moe::cluster_arrive();
    moe::cluster_wait();
}

}  // namespace

extern "C" __attribute__((visibility("default"))) int pair_run(int rounds, unsigned long long* out, void* stream) {
    pair_kernel<<<2, 32, 0, static_cast<cudaStream_t>(stream)>>>(rounds, out);
    return (int)cudaGetLastError();
}
extern "C" __attribute__((visibility("default"))) long long pair_polls() { return moe::kStallPolls; }
