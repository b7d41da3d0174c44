// pair_payload_probe.cu -- test helper, not part of libmoe: a cluster of two CTAs, in
// which a warp of CTA 1 writes a tile of its shared memory and arrives at a barrier of
// CTA 0 (csrc/tc.cuh), whose warp then reads the tile.  Every wait is bounded, so the
// kernel ends by itself.
#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "tc.cuh"

namespace {

constexpr int kWords = 512;

// out[0]: whether every wait ended; out[1]: rounds; out[2]: words that CTA 0 did not
// read as CTA 1 had written them in that round.
__global__ void __cluster_dims__(2, 1, 1) payload_kernel(int rounds, unsigned long long* out) {
    __shared__ uint64_t ready, taken;
    __shared__ uint32_t tile[kWords];
    __shared__ int gave_up;
    const uint32_t rank = moe::cluster_ctarank();
    const int lane = threadIdx.x;
    if (lane == 0) {
        moe::mbar_init(&ready, 1);
        moe::mbar_init(&taken, 1);
        moe::mbar_init_fence();
        gave_up = 0;
    }
    for (int i = lane; i < kWords; i += 32) tile[i] = 0xffffffffu;
    __syncwarp();
    moe::cluster_arrive();
    moe::cluster_wait();
    const uint32_t there = moe::peer_smem(moe::smem_u32(&ready), 0), back = moe::peer_smem(moe::smem_u32(&taken), 1);
    bool ok = true;
    unsigned long long done = 0, wrong = 0;
    for (int r = 0; ok && r < rounds; ++r) {
        if (rank == 1) {
            for (int i = lane; i < kWords; i += 32) tile[i] = (uint32_t)(r * kWords + i);
            __syncwarp();
            if (lane == 0) moe::mbar_arrive_cluster(there);
            ok = __all_sync(0xffffffffu, moe::mbar_wait_pair(&taken, r & 1, &gave_up));
        } else {
            ok = __all_sync(0xffffffffu, moe::mbar_wait_pair(&ready, r & 1, &gave_up));
            for (int i = lane; ok && i < kWords; i += 32)
                wrong += moe::ld_cluster_shared_u32(&tile[i], 1) != (uint32_t)(r * kWords + i);
            ++done;
            __syncwarp();
            if (lane == 0) moe::mbar_arrive_cluster(back);
        }
    }
    for (int off = 16; off > 0; off >>= 1) wrong += __shfl_xor_sync(0xffffffffu, wrong, off);
    if (rank == 0 && lane == 0) {
        out[0] = ok;
        out[1] = done;
        out[2] = wrong;
    }
    moe::cluster_arrive();
    moe::cluster_wait();
}

}  // namespace

extern "C" __attribute__((visibility("default"))) int payload_run(int rounds, unsigned long long* out, void* stream) {
    payload_kernel<<<2, 32, 0, static_cast<cudaStream_t>(stream)>>>(rounds, out);
    return (int)cudaGetLastError();
}
