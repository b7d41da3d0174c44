// experts.cu -- the experts' grouped products on E4M3 rows and weights.
//
//   y[r, n] = sum_b sa[r, b] sw[n / 128, b] sum_{i in block b} a[r, i] w[n, i]
//
// for every row r of expert p's window and every output n, with b the
// 128-element blocks of the inner dimension.  moe_experts_up computes gate and
// up outputs of the same 128 columns, h = silu(gate) up, and quantizes the 128
// values of each row as one group; moe_experts_down rounds y to bf16.
//
// Mapping.  One persistent CTA per SM walks tiles of 128 rows of one window by
// two 128-blocks of weight rows.  One thread loads operands by TMA, one issues
// tcgen05.mma (128 x 256 x 32, E4M3) into two TMEM accumulators, each of one
// 128-block of the inner dimension: the sum inside a block is the tensor core's,
// in fp32.  Scales are arbitrary fp32 values per row and block, so a block's
// sums cannot stay in TMEM: eight warps read them, multiply by sa * sw and add
// them up in registers (128 a thread).  A thread holds a row, and of it the same
// 64 columns of both blocks: gate and up meet in one thread, and the row's
// group maximum takes one exchange with one other warp.  Rows are the M operand
// whatever their number: an expert with few of them (a decode batch) is bound
// by its weights' bytes, and its product with 128 mostly empty rows fits into
// the time that they take to arrive.
//
// What bounds it (one GB300, back to back on new inputs).  Few rows an expert:
// HBM.  96 tokens x 8 over 256 experts of 7168 x 2048 (219 of them chosen, 6.4
// GB): 927 us, 6.9 TB/s, 1.02 of the measured copy peak.  4096 tokens, 288
// experts (8.8 GB): 1.31 ms from a cool GPU (0.98), 1.41 to 1.47 ms at its power
// limit, where the SM clock falls to 1.5 GHz.  Many rows: 98,304 rows over 64
// experts of 2048 x 1024, first product 330 us cool (2.5 PFLOP/s, 1.30 of the
// measured bf16 burst), 371 at the power limit; second 196 and 213.  There a
// block takes about 790 cycles, which no unit fills: the product needs 543 (alone
// on the SM; the tensor pipe counts 42 % active), the multiply-adds 256 of the
// FMA pipe, and reading and adding a block up takes a summing warp 420.  Taking
// the sums away shortens the first product to 214 us, so they are on the critical
// path; the other 370 cycles of a block, and about 2500 that a change of tile
// takes (the end of a tile runs in the summing warps, between two summing loops),
// have not been traced.  Reading TMEM is not what bounds it (loads of 16 columns
// cost 21 cycles one by one and do not slow the product).
//
// Measured and left out: 16 summing warps (434 against 402 us at the time);
// accumulators of 128 columns with two issuing threads (419 / 357); 32 or 64
// columns a TMEM load (364 / 352); one block of outputs a tile for small batches
// (one token's second product 27.8 / 26.1 us); row scales loaded four blocks at
// a time (345 / 336).
#include <cuda.h>

#include "maps.h"
#include "moe_internal.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "tc.cuh"
#include "windows.cuh"

namespace moe {
namespace {

constexpr int kMostExperts = 4096;
constexpr int kTileM = 128;        // rows of a tile (TMEM lanes)
constexpr int kTileN = 256;        // outputs of a tile: two 128-blocks of weight rows
constexpr int kRowBox = 32;        // rows per TMA box of the row operand
constexpr int kABytes = kTileM * kGroup;
constexpr int kBHalf = kGroup * kGroup;
constexpr int kStageBytes = kABytes + 2 * kBHalf;
constexpr int kSumWarps = 8;       // warps that scale and add up
constexpr int kTmaWarp = kSumWarps, kMmaWarp = kSumWarps + 1, kStoreWarp = kSumWarps + 2;
constexpr int kExpertsThreads = 32 * (kSumWarps + 4);  // three warpgroups
// Registers a thread, after setmaxnreg: 64,512 at launch (384 x 168) against
// 256 x 232 + 128 x 40 = 64,512.
constexpr int kSumRegs = 232, kOtherRegs = 40;
constexpr int kHalfN = kGroup / 2;  // columns of each 128-block that a summing warp owns

// The loading thread looks each tile up and leaves it in a ring for the other
// warps (a lookup costs about 1.5 k cycles of latency, which the summing warps
// cannot hide).  It runs ahead of the last reader by at most the operand
// buffers, the accumulators and a staged tile: 4 + 2 + 2 tiles of one block.
constexpr int kTileRing = 16;

// Finished rows wait in shared memory for the warps that copy them out, so
// that the summing warps can begin the next tile: columns of 128 bytes by
// kTileM rows, in the 128-byte swizzle of the boxes that TMA takes them out by
// (16-byte chunk c of row r lies at c ^ (r mod 8): no bank conflicts when a
// thread writes its row).  The bf16 tile takes the room of one operand buffer:
// three are enough, for the loads in flight at any time (21 MB over 152 SMs)
// are several times latency x bandwidth.
template <bool UP>
struct Layout {
    static constexpr int kStages = UP ? 4 : 3;      // operand buffers
    static constexpr int kOutColumns = UP ? 1 : 4;  // 128-byte columns of a tile's output
    static constexpr int kStagedBytes = kOutColumns * kTileM * kGroup;
    static constexpr int kBytes = kStages * kStageBytes + kStagedBytes;
};
constexpr int kOutBox = 32, kOutBoxSmall = 8;  // rows per TMA box of the output

__device__ __forceinline__ unsigned char* staged_chunk(unsigned char* staged, int column, int row, int chunk) {
    return staged + (column * kTileM + row) * kGroup + ((chunk ^ (row & 7)) << 4);
}

struct alignas(16) Barriers {
    uint64_t full[4], empty[4];          // operand buffers
    uint64_t acc_full[2], acc_empty[2];  // TMEM accumulators of one 128-block of K
    uint64_t staged, stage_free;         // finished rows
    uint64_t known[kTileRing];           // tiles[i] is written
    uint64_t drain;
    int4 tiles[kTileRing];  // expert, n, row, valid
    uint32_t tmem;
    int gave_up;
    int warp_total[kExpertsThreads / 32], warp_top[kExpertsThreads / 32];
    float maxima[2][kTileM];  // of the two halves of each row (Up)
};

struct Problem {
    int P, N, K;  // experts, outputs per row, inner size
    const float* sa;
    int sa_stride;
    const float* sw;
    const int32_t* offsets;
    int rows;
    uint8_t* h;
    float* hs;
    int hs_stride;
    uint16_t* out;
    int32_t* err;
};

// A tile is by two 128-blocks of its expert's weight rows: UP: gate block n and
// up block n; down: blocks 2n and 2n + 1 (the last one alone where their number
// is odd).

template <bool UP>
__global__ void __launch_bounds__(kExpertsThreads, 1)
experts_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_out_small,
               const Problem pr) {
    constexpr int kStages = Layout<UP>::kStages;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t skip = (1024u - (smem_u32(smem) & 1023u)) % 1024u;
    unsigned char* stages = smem + skip;
    unsigned char* staged = stages + kStages * kStageBytes;
    Barriers& b = *reinterpret_cast<Barriers*>(stages + Layout<UP>::kBytes);
    // The kernel has no other shared memory, so the base lies on a 1024-byte
    // boundary.  One that does not is refused, for there is no room to skip to
    // the next boundary.
    if (skip + Layout<UP>::kBytes + sizeof(Barriers) + (pr.P + 1) * sizeof(int) > dynamic_smem_bytes()) {
        grid_dependency_sync();  // no kernel behind this one starts before those in front of it are done
        if (threadIdx.x == 0) set_error(pr.err, MOE_DEVERR_STALL);
        return;
    }
    int* first_m = reinterpret_cast<int*>(&b + 1);  // [P + 1]
    volatile int* gave_up = &b.gave_up;
    // Uniform in a warp, and through the shuffle known to be: with elect_one it
    // lets the roles of one thread keep their addresses in uniform registers.
    const int warp = __shfl_sync(kFull, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(&b.full[s], 1);
                mbar_init(&b.empty[s], 1);
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(&b.acc_full[s], 1);
                mbar_init(&b.acc_empty[s], kSumWarps);
            }
            mbar_init(&b.staged, kSumWarps);
            mbar_init(&b.stage_free, 2);
            for (int i = 0; i < kTileRing; ++i) mbar_init(&b.known[i], 1);
            mbar_init(&b.drain, 1);
            b.gave_up = 0;
            mbar_init_fence();
        }
        __syncwarp();
        tmem_alloc_all(&b.tmem);
        tc_fence_before();
    } else if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_out);
        tma_prefetch_map(&map_out_small);
    }
    grid_dependency_sync();
    allow_dependents();
    const int blocks = pr.N / kGroup;                       // 128-blocks of outputs
    const int n_tiles = UP ? blocks : (blocks + 1) / 2;
    // its barriers publish the above
    const int m_total = scan_windows<kExpertsThreads, kTileM>(pr.offsets, pr.P, pr.rows, pr.err, first_m, b.warp_total,
                                                              b.warp_top, n_tiles, &b.tiles[0]);
    tc_fence_after();
    const uint32_t tmem = b.tmem;

    const int width = UP ? 2 * pr.N : pr.N;                 // weight rows per expert
    const int kb = pr.K / kGroup;
    const long long tiles = (long long)m_total * n_tiles;   // at most 2^31: checked by the host
    // Tile number j of this CTA, once the loading thread has left it in the
    // ring (wait_written: never an entry that it has not written).
    const auto tile_written = [&](uint32_t j) {
        return wait_written(MbarPhase{smem_u32(&b.known[j % kTileRing]), (j / kTileRing) & 1}, gave_up);
    };
    const auto tile_at = [&](uint32_t j) {
        const int4 v = *const_cast<const int4*>(&b.tiles[j % kTileRing]);
        return Tile{v.x, v.y, v.z, v.w};
    };
    // For a whole warp, the same answer in every lane (its TMEM loads and
    // barriers are the whole warp's).  After a wait has given up: an empty tile,
    // for which the warp sums, waits for and stores nothing, so that it still
    // passes the same barriers to the end.
    const auto known_tile = [&](uint32_t j) {
        const bool written = tile_written(j);
        const Tile t = tile_at(j);  // on its way while the lanes agree
        return __all_sync(kFull, written) ? t : Tile{0, 0, 0, 0};
    };

    if (warp >= kSumWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kTmaWarp && elect_one()) {
            int s = 0;
            uint32_t phase = 0, issued = 0;
            uint32_t used = 0x04040404u * (kTileM / kRowBox / 4);  // boxes holding something, 8 bits a buffer
            bool ok = true;
            TileWalk<kTileM> walk;
            uint32_t j = 0;
            for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++j) {
                // no tile is written any more, so none overwrites one that a
                // warp which runs on without waiting is reading
                if (!(ok = ok && *gave_up == 0)) break;
                Tile t;
                if (j == 0) {
                    const int4 v = b.tiles[0];
                    t = {v.x, v.y, v.z, v.w};
                    walk.p = t.p;
                } else {
                    t = walk.at((int)tile, n_tiles, first_m, pr.offsets, pr.P);
                    b.tiles[j % kTileRing] = make_int4(t.p, t.n, t.row, t.valid);
                }
                mbar_arrive(&b.known[j % kTileRing]);
                const int w0 = t.p * width + (UP ? t.n : 2 * t.n) * kGroup;
                const bool two = UP || 2 * t.n + 1 < blocks;
                const int w1 = UP ? w0 + pr.N : w0 + kGroup;
                const uint32_t boxes = (t.valid + kRowBox - 1) / kRowBox;
                const uint32_t weight_bytes = (two ? 2 : 1) * kBHalf;
                for (int k = 0; k < kb; ++k) {
                    if (!(ok = mbar_wait(&b.empty[s], phase ^ 1, gave_up))) break;
                    unsigned char* a = stages + s * kStageBytes;
                    // Rows of an earlier, fuller tile are cleared (by boxes past
                    // the end of the rows, which read nothing): their products
                    // would be thrown away, but not for free on a GPU that runs
                    // at its power limit.
                    const uint32_t held = (used >> (8 * s)) & 0xffu;
                    const uint32_t top = max(boxes, held);
                    used = (used & ~(0xffu << (8 * s))) | boxes << (8 * s);
                    mbar_expect_tx(&b.full[s], top * kRowBox * kGroup + weight_bytes);
                    tma_load_2d(a + kABytes, &map_w, k * kGroup, w0, &b.full[s]);
                    if (two) tma_load_2d(a + kABytes + kBHalf, &map_w, k * kGroup, w1, &b.full[s]);
                    for (uint32_t i = 0; i < top; ++i)
                        tma_load_2d(a + i * kRowBox * kGroup, &map_a, k * kGroup,
                                    i < boxes ? t.row + (int)(i * kRowBox) : pr.rows, &b.full[s]);
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) set_error(pr.err, MOE_DEVERR_STALL);
            // Leave only after the copies in flight have landed (or never will),
            // also where this thread was through before another wait gave up.
            const uint64_t t0 = now_ns();
            for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                while (!mbar_try(smem_u32(&b.full[i % kStages]), (i / kStages) & 1) && now_ns() - t0 < kStallNs) {
                }
        }
        if (warp == kMmaWarp && elect_one()) {
            int s = 0;
            uint32_t phase = 0, it = 0;
            bool ok = true;
            const uint64_t desc_a = umma_desc(stages), desc_w = umma_desc(stages + kABytes);
            uint32_t j = 0;
            for (long long tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x, ++j) {
                if (!UP && !(ok = tile_written(j))) break;
                const bool two = UP || 2 * tile_at(j).n + 1 < blocks;
                const uint32_t idesc = umma_idesc_e4m3(kTileM, two ? kTileN : kGroup);
                for (int k = 0; k < kb; ++k, ++it) {
                    const uint32_t buf = it & 1;
                    if (!(ok = mbar_wait(&b.full[s], phase, gave_up))) break;
                    if (!(ok = mbar_wait(&b.acc_empty[buf], ((it >> 1) & 1) ^ 1, gave_up))) break;
                    tc_fence_after();
                    const uint64_t da = desc_a + (uint32_t)s * (kStageBytes / 16);
                    const uint64_t dw = desc_w + (uint32_t)s * (kStageBytes / 16);
                    const uint32_t d = tmem + buf * kTileN;
#pragma unroll
                    for (int i = 0; i < kGroup / 32; ++i) {
                        if (i == 0)
                            umma_e4m3<false>(d, da, dw, idesc);
                        else
                            umma_e4m3<true>(d, da + 2 * i, dw + 2 * i, idesc);
                    }
                    umma_commit(&b.acc_full[buf]);
                    umma_commit(&b.empty[s]);
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) set_error(pr.err, MOE_DEVERR_STALL);
            umma_commit(&b.drain);  // the same for the products in flight
            const uint64_t t0 = now_ns();
            while (!mbar_try(smem_u32(&b.drain), 0) && now_ns() - t0 < kStallNs) {
            }
        }
        if (warp >= kStoreWarp) {
            // Copy finished rows out: one thread by TMA, whole boxes of 32 and 8
            // rows; the other warp the rows left over (a tile ends where its
            // window ends, and the next row is another expert's), 16 bytes a
            // lane.  (All rows by the two warps took 8.6 k cycles a bf16 tile,
            // a bulk copy for each row 11 k.)
            const int out_columns = Layout<UP>::kOutColumns;
            uint32_t j = 0;
            for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++j) {
                const Tile t = known_tile(j);
                const int columns = UP || 2 * t.n + 1 < blocks ? out_columns : out_columns / 2;
                if (t.valid > 0) mbar_pass(smem_u32(&b.staged), j & 1, gave_up);
                if (warp == kStoreWarp) {
                    if (elect_one()) {
                        const int x0 = t.n * (UP ? kGroup : kTileN);  // elements
                        for (int c = 0; c < columns; ++c) {
                            const int x = x0 + c * (UP ? kGroup : kGroup / 2);
                            const unsigned char* src = staged + c * kTileM * kGroup;
                            int r = 0;
                            for (; r + kOutBox <= t.valid; r += kOutBox)
                                tma_store_2d(&map_out, x, t.row + r, src + r * kGroup);
                            for (; r + kOutBoxSmall <= t.valid; r += kOutBoxSmall)
                                tma_store_2d(&map_out_small, x, t.row + r, src + r * kGroup);
                        }
                        bulk_commit();
                        bulk_wait_read();
                        mbar_arrive(&b.stage_free);
                    }
                    __syncwarp();
                } else {
                    const int from = t.valid & ~(kOutBoxSmall - 1), per_row = columns * 8;
                    for (int i = lane; i < (t.valid - from) * per_row; i += 32) {
                        const int r = from + i / per_row, c = i % per_row;
                        const uint4 v = *reinterpret_cast<const uint4*>(staged_chunk(staged, c >> 3, r, c & 7));
                        const size_t row = (size_t)(t.row + r) * pr.N;
                        st16(UP ? static_cast<void*>(pr.h + row + (size_t)t.n * kGroup + 16 * c)
                                : static_cast<void*>(pr.out + row + (size_t)t.n * kTileN + 8 * c),
                             v);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.stage_free);
                }
            }
            if (warp == kStoreWarp) {
                if (elect_one()) bulk_wait();
                __syncwarp();
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        // Summing warps: warp w reads TMEM lanes 32 (w mod 4) .. + 31 (a row a
        // thread) and of each 128-block the columns 64 (w / 4) .. + 63.
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t my_tmem = tmem + ((uint32_t)(quarter * 32) << 16) + half * kHalfN;
        const int in_tile = quarter * 32 + lane;
        uint32_t j = 0;
        Tile t = {0, 0, 0, 0};
        const float *sa = nullptr, *sw = nullptr;  // scales of the row and of the first 128-block
        int gap = 0;                               // from there to the second block's
        float ar = 0.0f, f0 = 0.0f, f1 = 0.0f;
        // Tile j and its first scales: loaded before the tile in front of it is
        // finished and stored, and needed after.
        const auto begin = [&]() {
            t = known_tile(j);
            sa = pr.sa + ((size_t)t.row + max(0, min(in_tile, t.valid - 1))) * pr.sa_stride;
            const int blk = UP ? t.n : 2 * t.n;
            sw = pr.sw + ((size_t)t.p * (width / kGroup) + blk) * kb;
            gap = UP ? blocks * kb : (blk + 1 < blocks ? kb : 0);
            ar = __ldg(sa);
            f0 = __ldg(sw);
            f1 = __ldg(sw + gap);
        };
        if (blockIdx.x < tiles) begin();
        // The two accumulators in turn: `buf` 0 or 1, `phase` the parity of their
        // barriers' phases, which flips after both.
        const uint32_t full_bar = smem_u32(&b.acc_full[0]), empty_bar = smem_u32(&b.acc_empty[0]);
        uint32_t buf = 0, phase = 0;
        // The accumulator is read: it may be written again.
        const auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(empty_bar + 8 * buf);
        };
        for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const bool busy = quarter * 32 < t.valid;  // the warp holds a row of the window
            const int steps = t.valid > 0 ? kb : 0;
            uint64_t acc[2][kHalfN / 2];
#pragma unroll
            for (int i = 0; i < kHalfN / 2; ++i) acc[0][i] = acc[1][i] = 0ull;
            // This loop is the compute-bound products' critical path, and every
            // instruction in it counts: unrolled four times, with constant
            // buffers and offsets, it is 25 % slower.
#pragma unroll 1
            for (int k = 0; k < steps; ++k) {
                const float s0 = ar * f0, s1 = ar * f1;
                if (k + 1 < kb) {  // the next block's scales, a block ahead
                    ar = __ldg(sa + k + 1);
                    f0 = __ldg(sw + k + 1);
                    f1 = __ldg(sw + gap + k + 1);
                }
                mbar_pass(full_bar + 8 * buf, phase, gave_up);
                tc_fence_after();
                if (busy) {
                    const uint32_t base = my_tmem + buf * kTileN;
                    uint32_t v[2][16];
                    tmem_load16(base, v[0]);
#pragma unroll
                    for (int c = 0; c < 2 * kHalfN / 16; ++c) {
                        tmem_wait_load(v[c & 1]);
                        if (c + 1 < 2 * kHalfN / 16)
                            tmem_load16(base + ((c + 1) / (kHalfN / 16)) * kGroup + ((c + 1) % (kHalfN / 16)) * 16,
                                        v[(c + 1) & 1]);
                        else
                            release();
                        const int h = c / (kHalfN / 16), c0 = (c % (kHalfN / 16)) * 8;
                        const uint32_t f = __float_as_uint(h == 0 ? s0 : s1);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[h][c0 + i] =
                                fma2(pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), pack2(f, f), acc[h][c0 + i]);
                    }
                } else {
                    release();
                }
                phase ^= buf;
                buf ^= 1;
            }
            const Tile now = t;
            const uint32_t parity = j & 1;
            ++j;
            if (tile + gridDim.x < tiles) begin();
            if constexpr (UP) {
                float amax = 0.0f;
                if (busy) {
#pragma unroll
                    for (int i = 0; i < kHalfN / 2; ++i) {
                        const float2 g = unpack2(acc[0][i]), u = unpack2(acc[1][i]);
                        const float x = gated(g.x, u.x), y = gated(g.y, u.y);
                        amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
                        acc[0][i] = pack2(__float_as_uint(x), __float_as_uint(y));
                    }
                }
                // the row's other 64 columns are with the warp 4 further (or back)
                if (now.valid > 0) mbar_pass(smem_u32(&b.stage_free), parity ^ 1, gave_up);
                b.maxima[half][in_tile] = amax;
                asm volatile("bar.sync %0, %1;" ::"r"(1 + quarter), "n"(64) : "memory");
                amax = fmaxf(amax, b.maxima[half ^ 1][in_tile]);
                if (busy) {
                    // a tiny group is scaled up first, so that 448 / amax stays finite
                    const float lift = amax < 0x1p-100f ? 0x1p64f : 1.0f;
                    const float inv = amax > 0.0f ? kE4M3Max / (amax * lift) : 0.0f;
#pragma unroll
                    for (int i = 0; i < kHalfN / 16; ++i) {
                        uint32_t q[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = unpack2(acc[0][8 * i + 2 * j]), y = unpack2(acc[0][8 * i + 2 * j + 1]);
                            q[j] = pack_e4m3x2(x.x * lift * inv, x.y * lift * inv) |
                                   pack_e4m3x2(y.x * lift * inv, y.y * lift * inv) << 16;
                        }
                        st_shared16(staged_chunk(staged, 0, in_tile, half * (kHalfN / 16) + i),
                                    make_uint4(q[0], q[1], q[2], q[3]));
                    }
                    if (half == 0 && in_tile < now.valid)
                        pr.hs[((size_t)now.row + in_tile) * pr.hs_stride + now.n] = amax / kE4M3Max;
                }
            } else {
                if (now.valid > 0) mbar_pass(smem_u32(&b.stage_free), parity ^ 1, gave_up);
                if (busy) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int i = 0; i < kHalfN / 8; ++i) {
                            uint32_t q[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 x = unpack2(acc[c][4 * i + j]);
                                q[j] = pack_bf16x2_rn(x.x, x.y);
                            }
                            st_shared16(staged_chunk(staged, 2 * c + half, in_tile, i),
                                        make_uint4(q[0], q[1], q[2], q[3]));
                        }
                    }
                }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.staged);
        }
        if (*gave_up && lane == 0) set_error(pr.err, MOE_DEVERR_STALL);
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_free_all(tmem);
    }
}

// ---- host side ----

template <bool UP>
int launch_experts(const Problem& pr, const uint8_t* a, const uint8_t* w, cudaStream_t s) {
    const int blocks = pr.N / kGroup, n_tiles = UP ? blocks : (blocks + 1) / 2;
    // The most row tiles any windows over these rows can have.
    const long long m_most = (long long)(pr.rows + kTileM - 1) / kTileM + min(pr.P, pr.rows);
    if (m_most * n_tiles > INT32_MAX) return MOE_ERR_SIZE;
    constexpr CUtensorMapDataType kByte = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    constexpr CUtensorMapDataType kOut = UP ? kByte : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const void* out = UP ? static_cast<const void*>(pr.h) : static_cast<const void*>(pr.out);
    CUtensorMap map_a, map_w, map_out, map_out_small;
    if (!tile_map(&map_a, kByte, a, (size_t)pr.rows, pr.K, kRowBox) ||
        !tile_map(&map_w, kByte, w, (size_t)pr.P * (UP ? 2 : 1) * pr.N, pr.K, kGroup) ||
        !tile_map(&map_out, kOut, out, (size_t)pr.rows, pr.N, kOutBox) ||
        !tile_map(&map_out_small, kOut, out, (size_t)pr.rows, pr.N, kOutBoxSmall))
        return MOE_ERR_CUDA;
    const size_t smem = Layout<UP>::kBytes + sizeof(Barriers) + (size_t)(pr.P + 1) * sizeof(int);
    // The same limit for every P, so that callers on several threads do not lower it for each other.
    constexpr size_t kMostSmem = Layout<UP>::kBytes + sizeof(Barriers) + (kMostExperts + 1) * sizeof(int);
    static_assert(kMostSmem <= 227 * 1024, "shared memory of one CTA");
    if (cudaFuncSetAttribute(experts_kernel<UP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    const int sms = sm_count();
    if (sms < 1) return MOE_ERR_CUDA;
    const unsigned grid = (unsigned)(m_most * n_tiles < sms ? m_most * n_tiles : sms);
    return launch_pdl(experts_kernel<UP>, dim3(grid), dim3(kExpertsThreads), smem, s, map_a, map_w, map_out,
                      map_out_small, pr) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_experts(const moe_experts* e) {
    if (e == nullptr || e->error_word == nullptr) return MOE_ERR_NULL;
    if (e->P < 1 || e->P > kMostExperts) return MOE_ERR_SIZE;
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
    const Problem pr = {e->P, e->I,     e->H, scales,   scale_stride, e->s13,  offsets,
                        rows, h,        h_scales, h_stride, nullptr,      e->error_word};
    return launch_experts<true>(pr, codes, e->w13, static_cast<cudaStream_t>(stream));
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
    const Problem pr = {e->P, e->H,    e->I,    h_scales, h_stride, e->s2,  offsets,
                        rows, nullptr, nullptr, 0,        out,      e->error_word};
    return launch_experts<false>(pr, h, e->w2, static_cast<cudaStream_t>(stream));
}
