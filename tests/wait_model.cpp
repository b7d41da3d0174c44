// wait_model.cpp -- the bounded wait of csrc/wait.h on the host, over phases
// whose polls and clock are counted: a poll of a phase that is not over sleeps
// as long as the hardware may let it, and reading the clock takes time too.
#include "wait.h"

namespace {

struct Sim {
    long long t = 0;  // ns
    long long polls = 0, looks = 0, reads = 0;
};

struct Phase {
    Sim* sim;
    long long ends;          // time at which the phase ends (negative: never)
    volatile int* gave_up;   // set by "another warp" ...
    long long other_gives_up;  // ... at this time (negative: never)
    bool done() const { return ends >= 0 && sim->t >= ends; }
    bool over() const {
        ++sim->looks;
        sim->t += 30;
        return done();
    }
    bool poll() const {
        ++sim->polls;
        sim->t += 45;
        if (!done()) {
            const long long wake = sim->t + moe::kPollNs;
            sim->t = ends >= 0 && ends < wake ? ends : wake;
        }
        if (other_gives_up >= 0 && sim->t >= other_gives_up) *gave_up = 1;
        return done();
    }
    uint64_t now() const {
        ++sim->reads;
        sim->t += 300;
        return (uint64_t)sim->t;
    }
};

// An mbarrier of a ring entry that has been written `uses` times: its current
// phase is number `uses`, and a wait on a parity is over while the current
// phase has the other one.
struct RingPhase {
    int uses;
    unsigned parity;
    uint64_t* clock;
    bool over() const { return (unsigned)(uses & 1) != parity; }
    bool poll() const {
        *clock += moe::kPollNs;
        return over();
    }
    uint64_t now() const { return *clock; }
};

}  // namespace

extern "C" {

long long wait_limit_ns() { return (long long)moe::kStallNs; }
long long wait_poll_ns() { return moe::kPollNs; }
long long wait_polls() { return moe::kStallPolls; }

// One wait, then `later` more on phases that never end, with the same flag.
// out: result, time, polls, clock reads of the first wait; time and polls of the
// later ones; how many of those returned true.
void wait_run(long long ends, long long other_gives_up, int later, long long* out) {
    volatile int gave_up = 0;
    Sim first;
    out[0] = moe::wait_bounded(Phase{&first, ends, &gave_up, other_gives_up}, &gave_up) ? 1 : 0;
    out[1] = first.t;
    out[2] = first.polls;
    out[3] = first.reads;
    Sim rest;
    out[6] = 0;
    for (int i = 0; i < later; ++i) out[6] += moe::wait_bounded(Phase{&rest, -1, &gave_up, -1}, &gave_up) ? 1 : 0;
    out[4] = rest.t;
    out[5] = rest.polls;
}

// A ring of `size` entries of which the writer filled numbers 0 .. written - 1
// and stopped: which of the entries 0 .. n - 1 a reader that takes one after the
// other counts as written.
void ring_run(int size, int written, int n, unsigned char* ok) {
    volatile int gave_up = 0;
    uint64_t clock = 0;
    for (int j = 0; j < n; ++j) {
        // what the entry's barrier shows a reader that is at number j: the
        // writer is ahead of it by less than a round, or has stopped
        int uses = 0;
        for (int w = j % size; w < written && w <= j; w += size) ++uses;
        ok[j] = moe::wait_written(RingPhase{uses, (unsigned)(j / size) & 1u, &clock}, &gave_up);
    }
}
}
