// route.cuh -- routing of one 32-token tile: the body every plan kernel
// runs per CTA (top-k by segment arg-max, gates from float pairs, replica
// pick, per-expert token masks, tile counts and in-tile ranks), with its key
// mapping and lane helpers.  Included by plan_kernels.cuh, after the trace
// buffers tr_route and tr_single are defined.
#pragma once

#include <climits>
#include <cstdint>

#include "dword.cuh"
#include "moe_internal.h"
#include "ptx.cuh"
#include "trace.cuh"

namespace moe {
namespace {

// The two largest keys of a lane that are not yet taken (bit r of `taken`
// marks slot r) and their slots (lower slot first among equal keys); k2 = 0
// if the lane has fewer than two such keys above 0.
template <int N>
__device__ __forceinline__ void lane_top2(const uint32_t (&key)[N], uint32_t taken, uint32_t& k1, int& r1,
                                          uint32_t& k2, int& r2) {
    k1 = 0u;
    r1 = 0;
    k2 = 0u;
    r2 = 0;
#pragma unroll
    for (int r = 0; r < N; ++r) {
        const uint32_t v = ((taken >> r) & 1u) ? 0u : key[r];
        if (v > k1) {
            k2 = k1;
            r2 = r1;
            k1 = v;
            r1 = r;
        } else if (v > k2) {
            k2 = v;
            r2 = r;
        }
    }
}

// Which kernel a route_tile call belongs to (its trace slice; the cluster
// plan keeps tile counts and ranks in shared memory instead of writing them).
constexpr int kRouteInRoute = 0, kRouteInSingle = 1, kRouteInCluster = 2;

#ifdef MOE_TRACE
// Stage stamps of route_tile go to the slice of the kernel that called it.
template <int WHERE>
__device__ __forceinline__ TraceSlice route_slice() {
    return WHERE == kRouteInRoute ? tr_route_t : tr_single_t;
}
#define ROUTE_MARK(stage) trace_mark(route_slice<WHERE>(), (stage))
#else
#define ROUTE_MARK(stage) ((void)0)
#endif

constexpr int kRouteThreads = 32 * kTileTokens;  // one warp per token of the tile


// Monotone map of finite floats onto uint32 (a < b  <=>  key(a) < key(b));
// -0 is folded onto +0 first, so equal values give equal keys.  Every finite
// value maps above 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    uint32_t b = __float_as_uint(f);
    if (b == 0x80000000u) b = 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Inverse of order_key (a -0 logit comes back as +0).
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// The gate of this thread's item (token itl = threadIdx.x / kp of the tile,
// j = threadIdx.x mod kp; 0 for a thread without an item), from the tile's
// selected logits sel_v [TT k] and the exp table in shared memory.
// Warp-collective in the first TT kp threads (whole warps).
template <int WHERE, int TT>
__device__ __forceinline__ float tile_gate(int T, int k, int t0, const float* sel_v, const float2* s_exp) {
    // ---- gates: g_j = exp(l_j - l_0) / sum_i exp(l_i - l_0), rounded once
    // to fp32.  Each token's k items sit in one segment of kp lanes (kp the
    // power of two >= k, so a segment never straddles a warp).  Each lane
    // forms d = l_j - l_0 exactly as a pair of floats and e_j = exp(d) as a
    // pair; a butterfly over the segment sums the pairs (every lane ends with
    // the same s: the pair sum is commutative); each lane divides e_j by s and
    // keeps the high float if Ziv's test shows it is the correctly rounded
    // quotient.  A token with an item the pairs cannot decide, or with
    // l_j - l_0 < -64, is redone in fp64 as e_j = exp(d) with e_0 = 1,
    // s = sum over j ascending and g_j = (float)(e_j / s). ----
    const int kp = k <= 1 ? 1 : 1 << (32 - __clz(k - 1));  // TT kp <= the CTA's threads
    const int itl = (int)threadIdx.x / kp;  // token within the tile (>= TT: no item)
    const int ij = (int)threadIdx.x - itl * kp;
    const int it = itl * k + ij;
    const bool item_ok = itl < TT && ij < k && t0 + itl < T;
    float g = 0.0f;
    bool slow = false;
    // Only the first TT kp threads hold items; warps past them skip the stage.
    // The test is per warp (TT kp may be below 32), so a warp that enters
    // enters whole and its full-mask shuffles see every lane.
    const bool gate_warp = ((int)threadIdx.x & ~31) < TT * kp;
    if (gate_warp) {
        dword::dw e = {0.0f, 0.0f};
        if (item_ok) {
            const dword::dw d = dword::two_sum(sel_v[it], -sel_v[itl * k]);
            if (d.h == 0.0f)
                e = {1.0f, 0.0f};  // j == 0, or a tie with the top logit
            else if (d.h >= -64.0f)
                e = dword::exp_dw(d.h, d.l, s_exp);
            else
                slow = true;  // far below the top logit (or not finite)
        }
        dword::dw s = e;
        for (int off = 1; off < kp; off <<= 1) {
            const dword::dw o = {__shfl_xor_sync(kFull, s.h, off), __shfl_xor_sync(kFull, s.l, off)};
            s = dword::dw_add(s, o);
        }
        if (item_ok && !slow) {
            const dword::dw q = dword::dw_div(e, s);
            g = q.h;
            slow = !dword::rounds_safely(q);
        }
    }
    ROUTE_MARK(2);
    const unsigned slow_lanes = gate_warp ? __ballot_sync(kFull, slow) : 0u;
    if (slow_lanes != 0u) {  // warp-uniform; rare
        const int seg = (int)(threadIdx.x & 31) & ~(kp - 1);
        const unsigned seg_bits = (kp == 32 ? 0xffffffffu : ((1u << kp) - 1u)) << seg;
        const bool redo = (slow_lanes & seg_bits) != 0u && item_ok;
        double e64 = 0.0;
        if (redo) e64 = (ij == 0) ? 1.0 : exp((double)sel_v[it] - (double)sel_v[itl * k]);
        double s64 = 0.0;
        for (int jj = 0; jj < k; ++jj) s64 += __shfl_sync(kFull, e64, seg + jj);
        if (redo) g = (float)(e64 / s64);
    }
    ROUTE_MARK(3);
    return g;
}

// moe_plan's router: keys are the logits, gates the softmax over the k
// selected ones (tile_gate).
struct TopkSoftmax {
    static constexpr bool kScored = false;
    static bool whole_warps(int, int) { return false; }
};

// moe_plan_routed's router.  Every quantity is binary32:
//   score s_e = 1 / (1 + exp(-l_e)), or exp(l_e - max l) / sum exp(l - max l)
//   choice c_e = s_e + bias_e; a group's score is the sum of its group_top
//   largest choices; the topk_group best groups stay (equal scores: the lower
//   group); the k largest choices in them are taken (equal: the lower id);
//   gate = s_e, over the sum of the k selected scores if renorm, times scale.
// The softmax's sum is that of its terms rounded to multiples of 2^-41
// (GridSum), which is exact in any order: the choices, and with them every
// integer the plan writes, are functions of the inputs alone, whatever the lanes
// per token.  (64-bit fixed point would do as well; its conversions cost 0.4 us
// more a plan of 96 tokens.)
struct ScoreRouter {
    static constexpr bool kScored = true;
    const float* bias;  // [E] or NULL
    float scale;
    bool sigmoid;
    int n_group, topk_group, group_top;
    bool renorm;
    // Whether the three-launch plan gives a token a whole warp whatever
    // route_lanes says.  Groups are compared across one (a lane a group).
    // Above 64 experts its rounds, with a ballot in place of a second
    // reduction, are the shorter ones (4096 tokens, 128 experts, top-8: 9.5 us
    // against 19.3 with 16 lanes); from 17 to 64 as long as every tile has an SM
    // to itself (softmax, top-6, 4096 tokens: 64 experts 7.8 us against 9.2 with 8
    // lanes, 32 experts 7.0 / 7.6, 20 experts 7.0 / 7.4; but 8192 tokens of 20
    // experts 8.6 / 8.0, 16384 of 64 16.6 / 14.1); up to 16 experts 8 lanes do
    // (4096 tokens 7.0 with a warp / 6.6, 16384 tokens 12.4 / 7.9).
    bool whole_warps(int T, int E) const {
        constexpr int kTilePerSm = 152 * kTileTokens;  // tokens
        return n_group > 1 || E > 64 || (E > 16 && T <= kTilePerSm);
    }

    // NaN (a NaN logit, or a row without a finite logit) counts as score 0.
    __device__ __forceinline__ float score(float l, float2 stat) const {
        const float s = sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - stat.x) / stat.y;
        return s == s ? s : 0.0f;
    }
};

// Keep the keys of the topk_group best groups and clear the others.  Lane
// `lane` of the whole warp holds the keys of experts [e0, e0 + st).
template <int EPL>
__device__ __forceinline__ void keep_best_groups(const ScoreRouter& ro, int E, int e0, int st, int lane,
                                                 uint32_t (&key)[EPL]) {
    const int size = E / ro.n_group;
    const int span = size / st;  // lanes per group
    if (span * st == size && (span & (span - 1)) == 0) {
        // Groups fall on whole lanes, a power of two of them (256 experts in 8
        // groups: 4 lanes each): all groups' two largest at once by a
        // butterfly over the group's lanes.
        uint32_t k1, k2;
        int r1, r2;
        lane_top2(key, 0u, k1, r1, k2, r2);
        for (int off = 1; off < span; off <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kFull, k1, off);
            const uint32_t o2 = __shfl_xor_sync(kFull, k2, off);
            k2 = max(min(k1, o1), max(k2, o2));
            k1 = max(k1, o1);
        }
        float v = key_value(k1);
        if (ro.group_top == 2) v += key_value(k2);
        const uint32_t mine = order_key(v);
        const int g = lane / span;
        int better = 0;
        for (int q = 0; q < ro.n_group; ++q) {
            const uint32_t o = __shfl_sync(kFull, mine, q * span);
            better += (o > mine || (o == mine && q < g)) ? 1 : 0;
        }
        if (better >= ro.topk_group) {
#pragma unroll
            for (int r = 0; r < EPL; ++r) key[r] = 0u;
        }
        return;
    }
    // Any other grouping: one group after the other, its largest keys by two
    // warp reductions; lane q keeps group q's score.
    uint32_t mine = 0u;
    for (int q = 0; q < ro.n_group; ++q) {
        uint32_t in[EPL];
#pragma unroll
        for (int r = 0; r < EPL; ++r) {
            const int e = e0 + r;
            in[r] = (e >= q * size && e < (q + 1) * size) ? key[r] : 0u;
        }
        uint32_t k1, k2;
        int r1, r2;
        lane_top2(in, 0u, k1, r1, k2, r2);
        const uint32_t m1 = __reduce_max_sync(kFull, k1);
        const int first = __ffs(__ballot_sync(kFull, k1 == m1)) - 1;
        const uint32_t m2 = __reduce_max_sync(kFull, lane == first ? k2 : k1);
        float v = key_value(m1);
        if (ro.group_top == 2) v += key_value(m2);
        if (lane == q) mine = order_key(v);
    }
    int better = 0;
    for (int q = 0; q < ro.n_group; ++q) {
        const uint32_t o = __shfl_sync(kFull, mine, q);
        better += (o > mine || (o == mine && q < lane)) ? 1 : 0;
    }
    const unsigned kept = __ballot_sync(kFull, lane < ro.n_group && better < ro.topk_group);
#pragma unroll
    for (int r = 0; r < EPL; ++r)
        if (e0 + r < E && !((kept >> ((e0 + r) / size)) & 1u)) key[r] = 0u;
}

// v[r] = src[e0 + r] for the r < st with e0 + r < n, else `other`.
template <int N>
__device__ __forceinline__ void load_run(const float* __restrict__ src, int n, int e0, int st, bool quads, float other,
                                         float (&v)[N]) {
#pragma unroll
    for (int r = 0; r < N; ++r) v[r] = other;
    if (N >= 4 && quads) {
#pragma unroll
        for (int r = 0; r + 3 < N; r += 4) {
            if (r < st && e0 + r < n) {
                const float4 q = __ldg(reinterpret_cast<const float4*>(src + e0 + r));
                v[r] = q.x;
                v[r + 1] = q.y;
                v[r + 2] = q.z;
                v[r + 3] = q.w;
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < N; ++r)
            if (r < st && e0 + r < n) v[r] = __ldg(src + e0 + r);
    }
}

// A sum of up to 1024 terms in [0, 1] that does not depend on their order: each
// term is cut into multiples of 2^-13, 2^-27 and 2^-41 (what is left, at most
// 2^-42, is dropped), and each kind is summed by itself.  A sum of one kind is a
// multiple of its grid and below 2^24 of it, so every addition is exact.  Adding
// and taking away 1.5 x 2^(23 - g) rounds to a multiple of 2^-g (Rump, Ogita and
// Oishi, "Accurate floating-point summation", SIAM J. Sci. Comput. 31(1), 2008).
struct GridSum {
    float hi = 0.0f, mid = 0.0f, lo = 0.0f;
    static __device__ __forceinline__ float cut(float& v, float c) {
        const float q = __fsub_rn(__fadd_rn(v, c), c);
        v = __fsub_rn(v, q);
        return q;
    }
    __device__ __forceinline__ void add(float e) {
        hi = __fadd_rn(hi, cut(e, 0x1.8p10f));
        mid = __fadd_rn(mid, cut(e, 0x1.8p-4f));
        lo = __fadd_rn(lo, cut(e, 0x1.8p-18f));
    }
    __device__ __forceinline__ void add_lane(int off) {  // the sum of lane ^ off
        hi = __fadd_rn(hi, __shfl_xor_sync(kFull, hi, off));
        mid = __fadd_rn(mid, __shfl_xor_sync(kFull, mid, off));
        lo = __fadd_rn(lo, __shfl_xor_sync(kFull, lo, off));
    }
    // to the nearest binary32, but for sums within 2^-47 of the middle of two
    __device__ __forceinline__ float value() const {
        const dword::dw t = dword::two_sum(mid, lo);
        const dword::dw u = dword::two_sum(hi, t.h);
        return __fadd_rn(u.h, __fadd_rn(u.l, t.l));
    }
};

// The keys of a scored router: the order keys of the choices of experts
// [e0, e0 + st) of one token (0 past E and for a token past T), groups
// applied.  A segment of L lanes holds a token; every lane of the warp takes
// part.  stat gets the softmax's (max, sum).
template <int EPL, int L>
__device__ __forceinline__ void scored_keys(const ScoreRouter& ro, const float* __restrict__ row, bool tok_ok, int E,
                                            int e0, int st, int sl, uint32_t (&key)[EPL], float2* stat) {
    float v[EPL];
    const bool quads = ((st | E) & 3) == 0;  // 16-byte aligned runs of four
    load_run(row, tok_ok ? E : 0, e0, st, quads, -INFINITY, v);
    // The biases travel with the logits where registers allow.
    constexpr int kEarly = EPL <= 8 ? EPL : 1;
    float early[kEarly];
    if (EPL <= 8 && ro.bias != nullptr) load_run(ro.bias, E, e0, st, quads, 0.0f, early);
    float2 ms = make_float2(0.0f, 1.0f);
    if (!ro.sigmoid) {
        float m = v[0];
#pragma unroll
        for (int r = 1; r < EPL; ++r) m = fmaxf(m, v[r]);
#pragma unroll
        for (int off = 1; off < L; off <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        GridSum sum;
#pragma unroll
        for (int r = 0; r < EPL; ++r) {
            const float e = expf(v[r] - m);  // 0 past E
            sum.add(e == e ? e : 0.0f);      // NaN: a NaN logit, or no finite one
        }
#pragma unroll
        for (int off = 1; off < L; off <<= 1) sum.add_lane(off);
        ms = make_float2(m, sum.value());
    }
    if (sl == 0) *stat = ms;
#pragma unroll
    for (int r = 0; r < EPL; ++r) {
        const int e = e0 + r;
        key[r] = 0u;
        if (tok_ok && r < st && e < E) {
            float c = ro.score(v[r], ms);
            if (ro.bias != nullptr) c += EPL <= 8 ? early[r < kEarly ? r : 0] : __ldg(ro.bias + e);
            key[r] = order_key(c == c ? c : -INFINITY);
        }
    }
    if (L == 32 && ro.n_group > 1) keep_best_groups(ro, E, e0, st, sl, key);
}

// The gate of this thread's item, from a scored router: the item's score
// (without a bias it is the selected choice itself), renormalised over the
// token's k items by a butterfly over their lanes.  Warp-collective in the
// first TT kp threads (whole warps).
template <int TT>
__device__ __forceinline__ float scored_gate(const ScoreRouter& ro, const float* __restrict__ logits, int T, int E,
                                             int k, int t0, const float* sel_v, const int32_t* sel_e,
                                             const float2* stat) {
    const int kp = k <= 1 ? 1 : 1 << (32 - __clz(k - 1));
    const int itl = (int)threadIdx.x / kp;
    const int ij = (int)threadIdx.x - itl * kp;
    const int it = itl * k + ij;
    float g = 0.0f;
    if (((int)threadIdx.x & ~31) < TT * kp) {
        if (itl < TT && ij < k && t0 + itl < T)
            g = ro.bias != nullptr ? ro.score(__ldg(logits + (size_t)(t0 + itl) * E + sel_e[it]), stat[itl])
                                   : sel_v[it];
        if (ro.renorm) {
            float sum = g;
            for (int off = 1; off < kp; off <<= 1) sum += __shfl_xor_sync(kFull, sum, off);
            g = sum > 0.0f ? g / sum : 0.0f;
        }
        g *= ro.scale;
    }
    return g;
}

// The gate of this thread's item for either router.  `head` is the start of
// the tile's shared memory: the exp table, or the scored router's (max, sum)
// per token.
template <int WHERE, int TT, class R>
__device__ __forceinline__ float router_gate(const R& router, const float* __restrict__ logits, int T, int E, int k,
                                             int t0, const float* sel_v, const int32_t* sel_e, const float2* head) {
    if constexpr (R::kScored)
        return scored_gate<TT>(router, logits, T, E, k, t0, sel_v, sel_e, head);
    else
        return tile_gate<WHERE, TT>(T, k, t0, sel_v, head);
}

// Route one tile of TT tokens (the body every plan kernel runs per CTA) with
// a CTA of THREADS = TT L threads: each token's top-k runs on a segment of L
// lanes (L = 32: a whole warp; 16 or 8 when the experts fit in at most 8 keys
// a lane, so that small expert counts do not occupy a whole warp per token).
// Tiles are 32 tokens (one mask word) except in the cluster plan, which
// spreads a small batch over more SMs with tiles of 8 or 16 tokens.
// Trace stages: 0 start, 1 top-k done, 2 gates from pairs done, 3 fp64
// fallback done, 4 replicas and masks done, 5 tile counts and ranks written.
template <int EPL, int WHERE, int THREADS, int TT, class R>  // EPL = logits per lane, at least ceil(E / L)
__device__ __forceinline__ void route_tile(const R& router, const float* __restrict__ logits, int T, int E, int P, int k,
                                           const int32_t* __restrict__ rep_off,
                                           const int32_t* __restrict__ rep_ids, int32_t* __restrict__ topk_e,
                                           float* __restrict__ gates, int32_t* __restrict__ phys,
                                           int32_t* __restrict__ tile_hist, int n_tiles,
                                           int32_t* __restrict__ local_rank, int32_t* __restrict__ err,
                                           unsigned char* smem, int tile) {
    constexpr int L = THREADS / TT;  // lanes per token
    static_assert(L == 8 || L == 16 || L == 32, "8, 16 or 32 lanes per token");
    static_assert(TT == 8 || TT == 16 || TT == 32, "8, 16 or 32 tokens per tile (bits of a mask word)");
    float2* s_exp = reinterpret_cast<float2*>(smem);                             // exp(m / 512) table
    float* sel_v = reinterpret_cast<float*>(s_exp + 2 * dword::kExpTableHalf + 1);  // [TT*k]
    int32_t* sel_e = reinterpret_cast<int32_t*>(sel_v + TT * k);  // [TT*k]
    int32_t* sel_p = sel_e + TT * k;                               // [TT*k]
    uint32_t* mask = reinterpret_cast<uint32_t*>(sel_p + TT * k);  // [P]
    int32_t* s_off = reinterpret_cast<int32_t*>(mask + P);                 // [E+1] replica CSR
    int32_t* s_ids = s_off + (E + 1);                                       // [P]

    ROUTE_MARK(0);
    // The exp table and the replica map go to shared memory by asynchronous
    // copies (no registers held, no wait) while the logits are loaded; they
    // are waited for before the barrier that ends the top-k.
    if (!R::kScored) {
        for (int i = threadIdx.x; i <= 2 * dword::kExpTableHalf; i += THREADS)
            cp_async8(s_exp + i, dword::kExpTable + i);
    }
    if (rep_off != nullptr) {
        for (int i = threadIdx.x; i <= E; i += THREADS) cp_async4(s_off + i, rep_off + i);
        for (int i = threadIdx.x; i < P; i += THREADS) cp_async4(s_ids + i, rep_ids + i);
    }
    const int tl = threadIdx.x / L;  // this segment's token within the tile
    const int sl = threadIdx.x % L;  // lane within the segment
    const int t0 = tile * TT;
    const int t = t0 + tl;

    // ---- top-k of token t: k rounds of segment arg-max, ties -> lower id ----
    // Logits (or a scored router's choices) become order-preserving unsigned
    // keys (-0 folded onto +0 so that equal floats give equal keys); lane s of
    // the segment holds experts s, s + L, s + 2L, ...; for a scored router
    // the run of st = ceil(E / L) experts from s st, so that a group of experts
    // is a run of lanes.  Each lane caches its two largest keys; a round
    // is one max-reduction of the lanes' first keys over the segment and one
    // min-reduction of the expert id among the lanes holding the maximum,
    // after which the winning lane marks the slot taken and promotes its
    // second key (rescanning only when it has none left).  Key 0 sits below
    // every finite logit and marks padding.  Lane j keeps the j-th winner and
    // its key, whose inverse is the selected logit.  Where a warp holds several
    // tokens every lane runs the rounds (a token past T has only padding keys
    // and writes nothing), so the segment butterflies below always see a
    // converged warp; a whole warp past T skips them (its lanes would rescan
    // their empty keys every round: 1.7 us of a one-token plan's 6).
    const bool tok_ok = t < T;
    if (L < 32 || tok_ok) {
        const float* row = logits + (size_t)(tok_ok ? t : t0) * E;
        uint32_t key[EPL];
        // expert of slot r: first + r * step
        const int step = R::kScored ? 1 : L;
        const int held = R::kScored ? (E + L - 1) / L : 0;
        const int first = R::kScored ? sl * held : sl;
        if constexpr (R::kScored) {
            scored_keys<EPL, L>(router, row, tok_ok, E, first, held, sl, key, s_exp + tl);
        } else {
#pragma unroll
            for (int r = 0; r < EPL; ++r) {
                const int e = r * L + sl;
                key[r] = (tok_ok && e < E) ? order_key(__ldg(row + e)) : 0u;
            }
        }
        uint32_t taken = 0u, k1, k2;
        int r1, r2;
        lane_top2(key, taken, k1, r1, k2, r2);
        uint32_t cand = (uint32_t)(first + r1 * step);
        int my_e = 0;
        uint32_t my_key = 0u;
        for (int j = 0; j < k; ++j) {
            uint32_t m;
            int win;
            if (L == 32 && R::kScored) {
                // Lanes hold ascending runs of experts, so of equal keys the
                // lowest lane's is the lowest expert: a ballot finds it (a third
                // less latency a round than a second redux.sync on the ids).
                m = __reduce_max_sync(kFull, k1);
                const int lane_w = __ffs(__ballot_sync(kFull, k1 == m)) - 1;
                win = (int)__shfl_sync(kFull, cand, lane_w);
            } else if (L == 32) {  // whole warp: redux.sync (26 cycles on GB300)
                m = __reduce_max_sync(kFull, k1);
                win = (int)__reduce_min_sync(kFull, (k1 == m) ? cand : (uint32_t)INT_MAX);
            } else {
                // A segment-masked redux.sync takes about 170 cycles here, so
                // the segment reduces (key, ~id) packed in 64 bits with one
                // xor butterfly: the largest key, then the smallest id.
                uint64_t kv = ((uint64_t)k1 << 32) | (uint64_t)(0xffffffffu - cand);
#pragma unroll
                for (int off = L / 2; off > 0; off >>= 1) {
                    const uint64_t o = __shfl_xor_sync(kFull, kv, off);
                    kv = o > kv ? o : kv;
                }
                m = (uint32_t)(kv >> 32);
                win = (int)(0xffffffffu - (uint32_t)kv);
            }
            if (win >= E) win = 0;  // only reachable with NaN logits (outside the domain)
            if (R::kScored ? (unsigned)(win - first) < (unsigned)held : sl == (win & (L - 1))) {
                taken |= 1u << r1;
                if (k2 != 0u) {
                    k1 = k2;
                    r1 = r2;
                    k2 = 0u;
                } else {
                    lane_top2(key, taken, k1, r1, k2, r2);
                }
                cand = (uint32_t)(first + r1 * step);
            }
            if (sl == j) {
                my_e = win;
                my_key = m;
            }
        }
        if (tok_ok && sl < k) {
            sel_v[tl * k + sl] = key_value(my_key);
            sel_e[tl * k + sl] = my_e;
        }
    }
    for (int p = threadIdx.x; p < P; p += THREADS) mask[p] = 0u;
    cp_async_wait_all();
    __syncthreads();
    ROUTE_MARK(1);

    const int kp = k <= 1 ? 1 : 1 << (32 - __clz(k - 1));  // TT kp <= THREADS (host's choice of L)
    const int itl = (int)threadIdx.x / kp;  // token within the tile (>= 32: no item)
    const int ij = (int)threadIdx.x - itl * kp;
    const int it = itl * k + ij;
    const bool item_ok = itl < TT && ij < k && t0 + itl < T;
    // The cluster plan computes the gates after its cluster barrier's arrive
    // (tile_gate there), where they hide behind the wait for the other CTAs.
    float g = 0.0f;
    if (WHERE != kRouteInCluster) g = router_gate<WHERE, TT>(router, logits, T, E, k, t0, sel_v, sel_e, s_exp);
    if (item_ok) {
        const int tt = t0 + itl;
        const int e = sel_e[it];
        int p = e;
        if (rep_off != nullptr) {
            const int lo = s_off[e];
            const int n = s_off[e + 1] - lo;
            if (n < 1 || lo < 0 || lo + n > P) {
                p = -1;
            } else {
                p = s_ids[lo + tt % n];
                if (p < 0 || p >= P) p = -1;
            }
            if (p < 0) set_error(err, MOE_DEVERR_REPLICA);
        }
        if (WHERE != kRouteInCluster) {  // the cluster plan stores these after its barrier
            const size_t o = (size_t)tt * k + ij;
            topk_e[o] = e;
            gates[o] = g;
            phys[o] = p;
        }
        sel_p[it] = p;
        if (p >= 0) {
            const uint32_t bit = 1u << itl;
            const uint32_t old = atomicOr(&mask[p], bit);
            if (old & bit) set_error(err, MOE_DEVERR_DUPLICATE);
        }
    }
    __syncthreads();
    ROUTE_MARK(4);

    // ---- tile histogram (expert-major) and in-tile ranks ----
    if (WHERE != kRouteInCluster) {
        for (int p = threadIdx.x; p < P; p += THREADS)
            tile_hist[(size_t)p * n_tiles + tile] = __popc(mask[p]);
        if (item_ok) {
            const int p = sel_p[it];
            local_rank[(size_t)(t0 + itl) * k + ij] = (p >= 0) ? __popc(mask[p] & ((1u << itl) - 1u)) : 0;
        }
    }
    ROUTE_MARK(5);
}

}  // namespace
}  // namespace moe
