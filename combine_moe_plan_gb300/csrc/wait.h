// wait.h -- the bounded wait of the experts' kernels, for any kind of phase: an
// mbarrier's (tc.cuh), or a counted one on the host (tests/wait_model.cpp).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_WAIT_FN __device__ __forceinline__
#else
#define MOE_WAIT_FN inline
#endif

// How long a wait may last once its clock runs.
#ifndef MOE_STALL_NS
#define MOE_STALL_NS 4000000000ull
#endif

namespace moe {

constexpr uint32_t kPollNs = 20000;  // a hint: a poll sleeps for about 4000 (33000 with acquire.cluster); it wakes when the phase ends
constexpr int kStallPolls = 256;     // polls before a wait's clock starts
constexpr uint64_t kStallNs = MOE_STALL_NS;

// Wait for `phase`: a look, then polls that may sleep.  A wait that is not over
// after kStallPolls polls (1 to 8 ms) starts a clock and gives up kStallNs
// later.  It then sets *gave_up, which every wait reads after each of its polls:
// those under way return false at their next poll, and each later one that is
// not over takes one poll.  The clock is not read at first because that takes
// several hundred cycles, which every wait that is not over at its first poll
// would pay; the flag is not read in front of a poll because that is 3 % of the
// products with many rows.
template <class Phase>
MOE_WAIT_FN bool wait_bounded(const Phase& phase, volatile int* gave_up) {
    if (phase.over()) return true;
    uint64_t t0 = 0;
    for (int i = 0;; ++i) {
        if (phase.poll()) return true;
        if (*gave_up) return false;
        if (i < kStallPolls) continue;
        if (i == kStallPolls)
            t0 = phase.now();
        else if (phase.now() - t0 > kStallNs)
            *gave_up = 1;
    }
}

// Wait until an entry of a ring is written: `phase` is that of the entry's
// barrier, whose parity stands for its uses in turn.  After a wait has given up
// the writer may have stopped anywhere, and the parity of a barrier that has been
// left behind says "over" again one round of the ring later, for an entry that
// was never written; so nothing counts as written from then on (and nothing is polled for).
template <class Phase>
MOE_WAIT_FN bool wait_written(const Phase& phase, volatile int* gave_up) {
    return (phase.over() || (*gave_up == 0 && wait_bounded(phase, gave_up))) && *gave_up == 0;
}

}  // namespace moe
