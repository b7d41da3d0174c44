// dense.cu -- the bf16 experts' grouped products and their gradients, for
// training: every expert's window of rows times its weights, forward and back.
//
//   up         g, u = x w13^T; h = silu(g) u; g and u kept as E4M3 codes
//   down       out = h w2^T
//   down_back  d = dout w2; back through the gates and the activation at the codes' values
//   up_back    dx = dgu w13
//   grad       dw = a^T b over the rows of a window
//
// Mapping.  Pairs of CTAs (clusters of two, one CTA per SM) walk tiles of 256 by
// 256 outputs, 128 rows in each CTA.  In each, one thread loads its half of both
// operands by TMA (64 inner elements a stage); one thread of the first CTA issues
// tcgen05.mma for both (256 x 256 x 16) into one of two TMEM accumulators; eight
// warps read the other accumulator, do what the product ends in, and send it out by
// TMA, each warp its own 32 rows in boxes of 128 bytes.  A CTA by itself (128 x 256)
// has to fetch 48 KB for 512 cycles of products, and an SM gets 64 bytes a cycle
// from L2: 768 cycles.  A pair fetches 32 KB a CTA.  Few rows an expert are another
// matter: there the weights' bytes from HBM are the time, and single CTAs, which keep
// more of them in flight (32 KB a stage instead of 16) and multiply fewer empty rows,
// are the faster form (PAIR false).
//   Rows are the M operand of every product with weights.  Weights are read as
// they lie: where the product runs over a row's inputs (up, down) they are a
// K-major operand, where it runs over the outputs (down_back, up_back) an MN-major
// one, and for grad both operands are: a window's rows are the inner dimension, of
// any number.  There the last stage of a window is loaded with zeros in front of the
// rows that are left (another expert's rows, or none, lie behind them: a NaN there must
// not meet a zero), and whole 16 rows of zeros are left out.  The zeros are TMA's, which
// fills what lies in front of its maps' second dimension (window_map): all of an operand
// is written by TMA and counted at the issuing CTA's barrier, so that nothing is handed
// from a thread of one CTA to one of the other.  (A warp that cleared the rows behind a
// window in shared memory would have to publish them to the other CTA, release.cluster,
// 1000 to 2200 cycles a tile: 1537 tokens over 44 experts in bf16 49.5 us that way, 40.7
// this way, and 50.2 with boxes of exactly the rows left and of zeros behind them, sixteen
// loads a tile.)
//
// What bounds it (one GB300; 98,304 rows over 64 experts of 2048 x 1024 unless named).
//   up, up_back: the tensor pipe, 92 and 91 % of it active, 544 and 543 cycles a stage
// of 512; from a cool GPU 480 and 472 us (1.72 and 1.75 PFLOP/s, the rows that fill the
// last tile of a window not counted), at the power limit, 1.4 to 1.5 GHz, 552 and 533.
// cuBLAS, 8192 cubed, on the same box: 1.88 and 1.72 PFLOP/s.
//   grad in fp32: 523 to 553 us cool, 575 to 629 hot (GPUs of two kinds of cooling).  Its stores (1.07 GB) cost 85 us of
// it, operands that miss L2 40: stores and loads get in each other's way between SM and
// L2 (43 bytes a cycle in, 7 out).  Stores through the load-store unit instead of TMA
// save nothing, 32 bytes a lane straight from registers cost 70 us more.
//   down_back: 363 to 371 us cool, 377 to 402 hot; half of the tensor pipe.  Finishing tiles costs 100
// us: codes in, three outputs out, 16 us of arithmetic.
//   Few rows an expert: HBM.  One token over 256 experts of 7168 x 2048, first product
// 77 us (69 at the copy peak), 96 tokens, second product 897 us (6.4 GB: 1.06 of the copy
// peak); 4096 tokens over 288, first product 2,623 (1.00).
//   More stages shorten everything (grad of 24,576 rows in bf16: 162 us with 6, 170 with
// 5, 218 with 3), so outputs have one box a warp.
//   Measured and left out: L2 prefetches of the operands 8 to 16 stages ahead (603 / 603
// us of grad, 420 / 410 of down_back); 16 finishing warps in down_back (493 / 413);
// its boxes 64 bytes wide with a stage more (448 / 413), or two of them (418 / 381); tiles
// looked up one ahead (no change).
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
constexpr int kTileN = 256, kStepK = 64;
constexpr int kHalfM = 128;                       // a CTA's rows (TMEM lanes)
__host__ __device__ constexpr int tile_m(bool pair) { return pair ? 2 * kHalfM : kHalfM; }
constexpr int kRowBox = 32;                       // rows per TMA box of a row operand and of an output
constexpr int kLine = 128;                        // bytes of a box's row
constexpr int kABytes = kHalfM * kLine;
// A stage: a CTA's rows, and the tile's columns or its half of them.
__host__ __device__ constexpr int stage_bytes(bool pair) { return kABytes + (pair ? kTileN / 2 : kTileN) * kLine; }
constexpr int kBlockBytes = kStepK * kLine;       // 64 outer elements of an operand
constexpr int kSumWarps = 8;                      // warps that finish tiles
constexpr int kTmaWarp = kSumWarps, kMmaWarp = kSumWarps + 1;
constexpr int kDenseThreads = 32 * (kSumWarps + 4);  // three warpgroups
// Registers a thread, after setmaxnreg: 64,512 at launch (384 x 168) against
// 256 x 216 + 128 x 72 = 64,512.
constexpr int kSumRegs = 216, kOtherRegs = 72;
constexpr int kBoxBytes = kRowBox * kLine;
constexpr int kMostStages = 6;
constexpr int kSmemLimit = 227 * 1024;

// The loading thread looks each tile up and leaves it in a ring for the other
// warps.  It runs ahead of the last reader by at most the stages, the
// accumulators and the tile being finished: every tile has at least one step.
constexpr int kTileRing = 16;

enum class Op { kUp, kDown, kDownBack, kUpBack, kGrad };

// Steps that are summed in TMEM before the sums go to registers.  The tensor cores
// cut their sums off instead of rounding them, which shortens a sum by about
// 2.4e-8 of it for every 16 terms (four times that where all terms have one sign).
// Every product is therefore summed 512 terms at a time (448 in grad, 768 in
// down_back, whose finishing takes longer than the products of two times 512 do), and
// those sums are added up in registers, rounded to nearest.  Results in bf16 need it as much as those
// in fp32: an inner size of 131,072 summed in one go came out short by 7.8e-4 on
// average, a fifth of a bf16 step.  It costs them nothing (98,304 rows over 64 experts
// of 2048 x 1024, up_back 469 us and 468 in one go, down 250 / 249).  The same rows,
// relative error of up_grad and of down_back's parts (torch's fp32 products: 4.2e-7 and
// 4.0e-7), and us of up_grad and down_back from a cool GPU:
//    256 terms  2.3e-7  2.8e-7  555  429
//    320        2.8e-7  3.2e-7  540  417
//    384        3.4e-7  3.7e-7  531  403
//    448        4.0e-7          523
//    512        4.5e-7  4.9e-7  523  379
//    768                6.9e-7       363
__host__ __device__ constexpr int chunk_of(Op op) { return op == Op::kDownBack ? 12 : op == Op::kGrad ? 7 : 8; }

struct alignas(16) Barriers {
    uint64_t full[kMostStages], empty[kMostStages];  // stages; full: both CTAs', in the first
    uint64_t acc_full[2], acc_empty[2];              // accumulators; empty: both CTAs', in the first
    uint64_t known[kTileRing];                       // tiles[i] is written
    // up .. up_back: expert, n, and of this CTA's half the first row and how many are valid;
    // grad: first row of this CTA's half in dw (-1: none), n, first row of the window, rows in it
    int4 tiles[kTileRing];
    uint32_t tmem;
    int gave_up;
    int warp_total[kDenseThreads / 32], warp_top[kDenseThreads / 32];
};

// Boxes of outputs that a finishing warp holds, and the stages beside them: 224 KB in
// all.  A stage more is worth more than a box more where the boxes of a tile can
// wait for one another (grad of 98,304 rows: 602 us with 6 stages and 1 box, 621
// with 5 and 2, 661 with 4 and 3); down_back's three leave together.
__host__ __device__ constexpr int boxes_of(Op op) { return op == Op::kDownBack ? 3 : 1; }
__host__ __device__ constexpr int stages_of(Op op, bool pair) {
    return (224 * 1024 - kSumWarps * boxes_of(op) * kBoxBytes) / stage_bytes(pair);
}
__host__ __device__ constexpr size_t smem_bytes(Op op, bool pair, int stages, int P) {
    return (size_t)stages * stage_bytes(pair) + kSumWarps * boxes_of(op) * kBoxBytes + sizeof(Barriers) + (size_t)(P + 1) * sizeof(int);
}
static_assert(stages_of(Op::kDown, true) == kMostStages, "stages that the barriers are for");
static_assert(smem_bytes(Op::kDown, true, kMostStages, 512) <= kSmemLimit, "every stage up to 512 experts and more");
static_assert(smem_bytes(Op::kDown, true, kMostStages - 1, kMostExperts) <= kSmemLimit, "shared memory of one CTA");

struct Problem {
    int P, N, K;  // experts, outputs a row, inner size; grad: columns of b and of a
    const int32_t* offsets;
    int rows;
    uint16_t* out;     // up: h; down, up_back: the rows; down_back: hg
    uint16_t* dgu;     // down_back
    uint8_t* codes;    // up: out, or NULL; down_back: in
    float* scales;
    int scale_stride;
    const float* row_gates;
    float* parts;
    void* dw;
    int grad;
    int stages;
    int32_t* err;
};

// ---- finishing a tile: what one warp does with 32 rows by 128 columns ----

// A lane's 128 sums, in pairs: of its row 64 columns from accumulator column c0
// and 64 from c1.
struct Sums {
    uint64_t v[64];
    __device__ __forceinline__ float2 at(int pair) const { return unpack2(v[pair]); }
};

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(__float_as_uint(v), __float_as_uint(v)); }

template <bool FIRST>
__device__ __forceinline__ void take_sums(Sums& s, uint32_t c0, uint32_t c1) {
    uint32_t v[2][16];
    tmem_load16(c0, v[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        tmem_wait_load(v[c & 1]);
        if (c + 1 < 8) tmem_load16((c + 1 < 4 ? c0 : c1) + ((c + 1) & 3) * 16, v[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t pair = pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]);
            s.v[8 * c + i] = FIRST ? pair : add2(s.v[8 * c + i], pair);
        }
    }
}

// A warp's boxes of outputs on their way out: 32 rows of 128 bytes in shared
// memory, 16-byte chunk c of row r at c ^ (r mod 8) (the 128-byte swizzle: no bank
// conflicts when a lane writes its row).
struct Boxes {
    unsigned char* base;  // of this warp
    int lane;

    // The boxes sent have been read, by TMA or by this warp.
    __device__ __forceinline__ void wait() const {
        if (elect_one()) bulk_wait_read();
        __syncwarp();
    }
    __device__ __forceinline__ void put(int box, int chunk, uint4 v) const { put_at(base + box * kBoxBytes, chunk, v); }
    __device__ __forceinline__ void put_at(unsigned char* box, int chunk, uint4 v) const {
        st_shared16(box + lane * kLine + ((chunk ^ (lane & 7)) << 4), v);
    }
    __device__ __forceinline__ void put_row(int box, int row, int chunk, uint4 v) const {
        st_shared16(base + box * kBoxBytes + row * kLine + ((chunk ^ (row & 7)) << 4), v);
    }
    __device__ __forceinline__ uint4 get(int box, int chunk) const {
        return *reinterpret_cast<const uint4*>(base + box * kBoxBytes + lane * kLine + ((chunk ^ (lane & 7)) << 4));
    }
    // This lane's part of the boxes may be read by TMA.
    __device__ __forceinline__ void ready() const {
        fence_async_shared();
        __syncwarp();
    }
    // A box to (x, row) of the map: by TMA if all 32 rows are wanted, else the
    // first `rows` of them 16 bytes a lane, to `at` and on by `pitch` bytes a row
    // (a window ends here, and the next row is another expert's).
    __device__ __forceinline__ void send(int box, const CUtensorMap* map, int x, int row, int rows, void* at, size_t pitch) const {
        const unsigned char* from = base + box * kBoxBytes;
        if (rows < kRowBox) {
            for (int i = lane; i < rows * 8; i += 32) {
                const int r = i >> 3, c = i & 7;
                const uint4 v = *reinterpret_cast<const uint4*>(from + r * kLine + ((c ^ (r & 7)) << 4));
                st16(static_cast<unsigned char*>(at) + r * pitch + c * 16, v);
            }
            __syncwarp();
            return;
        }
        if (elect_one()) {
            tma_store_2d(map, x, row, from);
            bulk_commit();
        }
        __syncwarp();
    }
};

// up: a lane has 64 gate and the same 64 up columns of its row; the other 64 are
// with the warp of the other half, and so the groups' maxima are exchanged (through
// the boxes: shared memory of their own would cost a stage from 90 experts on).  The
// codes of a row's 128 gate columns leave from one warp's box, those of its up
// columns from the other's.
__device__ __forceinline__ void finish_up(const Problem& pr, const CUtensorMap* map_out, const CUtensorMap* map_codes,
                                          const Boxes& box, unsigned char* other, const Sums& s, int quarter, int half,
                                          int n, int row, int rows) {
    float top_g = 0.0f, top_u = 0.0f;
    if (rows > 0) {
        box.wait();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 g = s.at(4 * c + i), u = s.at(32 + 4 * c + i);
                h[i] = pack_bf16x2_rn(gated(g.x, u.x), gated(g.y, u.y));
                top_g = fmaxf(top_g, fmaxf(fabsf(g.x), fabsf(g.y)));
                top_u = fmaxf(top_u, fmaxf(fabsf(u.x), fabsf(u.y)));
            }
            box.put(0, c, make_uint4(h[0], h[1], h[2], h[3]));
        }
        const int x = n * kGroup + half * 64;
        box.ready();
        box.send(0, map_out, x, row, rows, pr.out + (size_t)row * pr.N + x, (size_t)pr.N * 2);
    }
    if (pr.codes == nullptr) return;
    // Both warps come here for every tile, rows or none.
    box.wait();
    reinterpret_cast<float2*>(box.base)[box.lane] = make_float2(top_g, top_u);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + quarter), "n"(64) : "memory");  // both maxima, both boxes free
    const float2 tops = reinterpret_cast<const float2*>(other)[box.lane];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + quarter), "n"(64) : "memory");  // both read
    if (rows > 0) {
        top_g = fmaxf(top_g, tops.x);
        top_u = fmaxf(top_u, tops.y);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float top = m == 0 ? top_g : top_u;
            // a tiny group is scaled up first, so that 448 / top stays finite
            const float lift = top < 0x1p-100f ? 0x1p64f : 1.0f;
            const float inv = top > 0.0f ? kE4M3Max / (top * lift) : 0.0f;
            unsigned char* to = half == m ? box.base : other;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = s.at(32 * m + 8 * c + 2 * i), b = s.at(32 * m + 8 * c + 2 * i + 1);
                    q[i] = pack_e4m3x2(a.x * lift * inv, a.y * lift * inv) |
                           pack_e4m3x2(b.x * lift * inv, b.y * lift * inv) << 16;
                }
                box.put_at(to, half * 4 + c, make_uint4(q[0], q[1], q[2], q[3]));
            }
        }
        fence_async_shared();
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + quarter), "n"(64) : "memory");
    if (rows > 0) {
        const int xc = half * pr.N + n * kGroup;
        box.send(0, map_codes, xc, row, rows, pr.codes + (size_t)row * 2 * pr.N + xc, (size_t)pr.N * 2);
        if (box.lane < rows)
            pr.scales[(size_t)(row + box.lane) * pr.scale_stride + half * (pr.N / kGroup) + n] =
                (half == 0 ? top_g : top_u) / kE4M3Max;
    }
}

// down, up_back, and grad in bf16: two boxes of 64 columns.
__device__ __forceinline__ void finish_rows(const CUtensorMap* map, const Boxes& box, const Sums& s, int x, int row, int rows,
                                            uint16_t* out, int width) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        box.wait();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = s.at(32 * b + 4 * c + i);
                q[i] = pack_bf16x2_rn(v.x, v.y);
            }
            box.put(0, c, make_uint4(q[0], q[1], q[2], q[3]));
        }
        box.ready();
        box.send(0, map, x + b * 64, row, rows, out + (size_t)row * width + x + b * 64, (size_t)width * 2);
    }
}

// Two E4M3 codes as floats.
__device__ __forceinline__ uint64_t unpack_e4m3x2(uint32_t w) {
    uint32_t h, lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(h));
    return pack2(lo, hi);
}

__device__ __forceinline__ uint32_t pack_bf16(uint64_t pair) {
    const float2 v = unpack2(pair);
    return pack_bf16x2_rn(v.x, v.y);
}

// What finishing a tile of down_back needs of a lane's row besides the codes: loaded
// while the tile is summed.
struct RowScalars {
    float gate, sg, su;
};
__device__ __forceinline__ RowScalars row_scalars(const Problem& pr, size_t row, int blk) {
    const float* scales = pr.scales + row * pr.scale_stride + blk;
    return {__ldg(pr.row_gates + row), __ldg(scales), __ldg(scales + pr.N / kGroup)};
}

// 64 columns of the codes of this warp's 32 rows (gate's, then up's): four lanes a
// row, so that a load touches 8 lines and not 32.  Lanes past `rows` repeat the last row.
struct CodeLines {
    uint4 v[8];
};
__device__ __forceinline__ CodeLines load_codes(const Problem& pr, int column, int row, int rows, int lane) {
    CodeLines c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t r = (size_t)row + min(8 * i + (lane >> 2), rows - 1);
        const uint8_t* p = pr.codes + r * 2 * pr.N + column + (lane & 3) * 16;
        c.v[i] = ld_stream16(p);
        c.v[4 + i] = ld_stream16(p + pr.N);
    }
    return c;
}

// down_back: a lane has one 128-group of its row, whose scales and sum are its own.
// The codes are in L2 by now (the loading thread saw to it when it began the tile) and
// go to their lanes through the third box: a lane's own 128 bytes of it are its row's
// 64 gate and 64 up codes.
//   s = sigmoid(g), h = g s u, hg = gate h, du = gate d g s, dg = gate d u (s + g s (1 - s))
__device__ __forceinline__ void finish_down_back(const Problem& pr, const CUtensorMap* map_hg, const CUtensorMap* map_dgu,
                                                 const Boxes& box, const Sums& d, const RowScalars& rs, int blk, int row,
                                                 int rows) {
    const size_t mine = (size_t)row + min(box.lane, rows - 1);
    const uint64_t gate = both(rs.gate), sg = both(rs.sg), su = both(rs.su);
    const uint64_t one = both(1.0f), minus_one = both(-1.0f);
    uint64_t sum = 0ull;
    CodeLines lines = load_codes(pr, blk * kGroup, row, rows, box.lane);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        box.wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) box.put_row(2, 8 * (i & 3) + (box.lane >> 2), (i >> 2) * 4 + (box.lane & 3), lines.v[i]);
        __syncwarp();
        uint4 cg[4], cu[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) cg[i] = box.get(2, i), cu[i] = box.get(2, 4 + i);
        __syncwarp();
        if (b == 0) lines = load_codes(pr, blk * kGroup + 64, row, rows, box.lane);
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // 8 columns
            const uint4 pg = cg[c >> 1], pu = cu[c >> 1];
            const uint32_t wg[2] = {c & 1 ? pg.z : pg.x, c & 1 ? pg.w : pg.y};
            const uint32_t wu[2] = {c & 1 ? pu.z : pu.x, c & 1 ? pu.w : pu.y};
            uint32_t dg[4], du[4], hg[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint64_t g = mul2(unpack_e4m3x2(wg[q >> 1] >> (16 * (q & 1))), sg);
                const uint64_t u = mul2(unpack_e4m3x2(wu[q >> 1] >> (16 * (q & 1))), su);
                const float2 gs = unpack2(g);
                const uint64_t sig = pack2(__float_as_uint(sigmoid(gs.x)), __float_as_uint(sigmoid(gs.y)));
                const uint64_t dd = d.v[32 * b + 4 * c + q], dh = mul2(gate, dd);
                const uint64_t silu = mul2(g, sig), h = mul2(silu, u);
                sum = fma2(dd, h, sum);
                hg[q] = pack_bf16(mul2(gate, h));
                du[q] = pack_bf16(mul2(dh, silu));
                dg[q] = pack_bf16(mul2(mul2(dh, u), fma2(silu, fma2(sig, minus_one, one), sig)));
            }
            box.put(0, c, make_uint4(dg[0], dg[1], dg[2], dg[3]));
            box.put(1, c, make_uint4(du[0], du[1], du[2], du[3]));
            box.put(2, c, make_uint4(hg[0], hg[1], hg[2], hg[3]));
        }
        const int x = blk * kGroup + b * 64;
        const size_t wide = (size_t)2 * pr.N;
        box.ready();
        box.send(0, map_dgu, x, row, rows, pr.dgu + row * wide + x, wide * 2);
        box.send(1, map_dgu, pr.N + x, row, rows, pr.dgu + row * wide + pr.N + x, wide * 2);
        box.send(2, map_hg, x, row, rows, pr.out + (size_t)row * pr.N + x, (size_t)pr.N * 2);
    }
    const float2 total = unpack2(sum);
    if (box.lane < rows) pr.parts[mine * (pr.N / kGroup) + blk] = total.x + total.y;
}

// grad in fp32: four boxes of 32 columns, one after the other.
__device__ __forceinline__ void finish_grad(const CUtensorMap* map, const Boxes& box, const Sums& s, int x, int row, bool add) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        box.wait();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float2 u = s.at(16 * b + 2 * c), v = s.at(16 * b + 2 * c + 1);
            box.put(0, c, make_uint4(__float_as_uint(u.x), __float_as_uint(u.y), __float_as_uint(v.x), __float_as_uint(v.y)));
        }
        box.ready();
        if (elect_one()) {
            if (add)
                tma_add_2d(map, x + b * 32, row, box.base);
            else
                tma_store_2d(map, x + b * 32, row, box.base);
            bulk_commit();
        }
        __syncwarp();
    }
}

template <Op OP, bool PAIR>
__global__ void __launch_bounds__(kDenseThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_a_small,
             const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_out2,
             const __grid_constant__ CUtensorMap map_codes, const Problem pr) {
    constexpr bool kGrad = OP == Op::kGrad;
    constexpr bool kBMn = OP == Op::kDownBack || OP == Op::kUpBack || kGrad;  // B lies MN-major
    constexpr int kChunk = chunk_of(OP), kWarpBytes = boxes_of(OP) * kBoxBytes;
    constexpr int kTileM = tile_m(PAIR), kStageBytes = stage_bytes(PAIR);
    static_assert(PAIR || (OP != Op::kDownBack && !kGrad), "forms that are not needed");
    extern __shared__ __align__(1024) unsigned char smem[];
    const int stages = pr.stages;
    // The kernel has no other shared memory, so the base lies on a 1024-byte
    // boundary.  One that does not is refused.
    if ((smem_u32(smem) & 1023u) != 0 || smem_bytes(OP, PAIR, stages, pr.P) > dynamic_smem_bytes()) {
        grid_dependency_sync();  // no kernel behind this one starts before those in front of it are done
        if (threadIdx.x == 0) set_error(pr.err, MOE_DEVERR_STALL);
        return;
    }
    unsigned char* staging = smem + stages * kStageBytes;
    Barriers& b = *reinterpret_cast<Barriers*>(staging + kSumWarps * kWarpBytes);
    int* first_m = reinterpret_cast<int*>(&b + 1);  // [P + 1]
    volatile int* gave_up = &b.gave_up;
    // Uniform in a warp, and through the shuffle known to be.
    const int warp = __shfl_sync(kFull, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const int pair = PAIR ? blockIdx.x >> 1 : blockIdx.x, pairs = PAIR ? gridDim.x >> 1 : gridDim.x;  // of those that share tiles

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(&b.full[s], PAIR ? 2 : 1);
                mbar_init(&b.empty[s], 1);
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(&b.acc_full[s], 1);
                mbar_init(&b.acc_empty[s], (PAIR ? 2 : 1) * kSumWarps);
            }
            for (int i = 0; i < kTileRing; ++i) mbar_init(&b.known[i], 1);
            b.gave_up = 0;
            mbar_init_fence();
        }
        __syncwarp();
        if (PAIR)
            tmem_alloc_all_pair(&b.tmem);
        else
            tmem_alloc_all(&b.tmem);
        tc_fence_before();
    } else if (warp == kTmaWarp && lane == 0) {
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_a_small);
        tma_prefetch_map(&map_b);
        tma_prefetch_map(&map_out);
        tma_prefetch_map(&map_out2);
    }
    if (PAIR) cluster_arrive();
    grid_dependency_sync();
    allow_dependents();
    const int blocks = pr.N / kGroup;  // 128-blocks of outputs
    const int n_tiles = OP == Op::kUp ? blocks : (blocks + 1) / 2;
    // its barriers publish the above to this CTA, the cluster's to the other
    const int m_total = scan_windows<kDenseThreads, kGrad ? kStepK : kTileM>(
        pr.offsets, pr.P, pr.rows, pr.err, first_m, b.warp_total, b.warp_top);
    if (PAIR) cluster_wait();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    // at most 2^31: checked by the host
    const int m_tiles = (pr.K + kTileM - 1) / kTileM;  // grad
    const long long tiles = (long long)(kGrad ? pr.P * m_tiles : m_total) * n_tiles;

    // Tile number j of this CTA, once the loading thread has left it in the ring.
    const auto tile_written = [&](uint32_t j) {
        return wait_written(MbarPhase{smem_u32(&b.known[j % kTileRing]), (j / kTileRing) & 1}, gave_up);
    };
    const auto tile_at = [&](uint32_t j) { return *const_cast<const int4*>(&b.tiles[j % kTileRing]); };
    // Steps of a tile along the inner dimension.  A window without rows has one,
    // of zeros (past the end of the rows), so that its gradient is zeros like any other's.
    const auto steps_of = [&](const int4& t) { return kGrad ? max(1, (t.w + kStepK - 1) / kStepK) : pr.K / kStepK; };

    // grad: tile number `tile` as the ring has it (of this CTA's half).
    const auto grad_tile = [&](long long tile) {
        const int mn = (int)(tile / n_tiles), p = mn / m_tiles;
        const int m0 = (mn - p * m_tiles) * kTileM + rank * kHalfM;
        const int lo = pr.offsets[p], count = first_m[p + 1] > first_m[p] ? pr.offsets[p + 1] - lo : 0;
        return make_int4(m0 < pr.K ? p * pr.K + m0 : -1, (int)(tile - (long long)mn * n_tiles), count > 0 ? lo : pr.rows,
                         count);
    };

    if (warp >= kSumWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTmaWarp) {
        if (elect_one()) {
            int s = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            TileWalk<kTileM> walk;
            const uint32_t full = PAIR ? peer_smem(smem_u32(&b.full[0]), 0) : 0;
            uint32_t j = 0;
            for (long long tile = pair; tile < tiles; tile += pairs, ++j) {
                // no tile is written any more, so none overwrites one that a
                // warp which runs on without waiting is reading
                if (!(ok = ok && *gave_up == 0)) break;
                int4 t;
                int m0 = 0, p = 0;
                if constexpr (kGrad) {
                    t = grad_tile(tile);
                    m0 = (int)((tile / n_tiles) % m_tiles) * kTileM + rank * kHalfM;
                } else {
                    const Tile w = walk.at((int)tile, n_tiles, first_m, pr.offsets, pr.P);
                    p = w.p;
                    t = make_int4(p, w.n, w.row + rank * kHalfM, max(0, min(kHalfM, w.valid - rank * kHalfM)));
                }
                b.tiles[j % kTileRing] = t;
                mbar_arrive(&b.known[j % kTileRing]);
                const bool two = OP == Op::kUp || 2 * t.y + 1 < blocks;
                const int steps = steps_of(t);
                if (OP == Op::kDownBack && t.w > 0)
                    for (int i = 0; i < (two ? 4 : 2); ++i)  // gate and up columns of its blocks
                        tma_prefetch_2d(&map_codes, (i & 1) * pr.N + (2 * t.y + (i >> 1)) * kGroup, t.z);
                // The columns of this CTA begin at n0.  Of a pair each loads 128; with one
                // block of 128 outputs left it takes 64 of each.
                const int n0 = OP == Op::kUp ? t.y * kGroup + rank * pr.N : t.y * kTileN + rank * (two ? kGroup : 64);
                // A single CTA loads a whole box of rows, or as many small ones as hold any: a
                // few rows an expert should not cost 16 KB a stage.  A pair clears the boxes
                // that hold none (by boxes past the end of the rows, which read nothing): the
                // products of what an earlier tile left there would be thrown away, but not for
                // free on a GPU that runs at its power limit (up_back of 98,304 rows 538 us / 546).
                const int small = !kGrad && t.w < kHalfM ? (t.w + kRowBox - 1) / kRowBox : 0;
                const bool few = !PAIR && t.w <= kHalfM / 2;
                const uint32_t bytes = kStageBytes - (few ? kABytes - small * kBoxBytes : 0) - (PAIR || two ? 0 : kGroup * kLine);
                for (int k = 0; k < steps; ++k) {
                    if (!(ok = mbar_wait(&b.empty[s], phase ^ 1, gave_up))) break;
                    unsigned char *pa = smem + s * kStageBytes, *pb = pa + kABytes;
                    const int inner = k * kStepK;
                    if constexpr (PAIR) {
                        const uint32_t bar = full + 8 * s;
                        mbar_expect_tx_cluster(bar, bytes);
                        if constexpr (kGrad) {
                            const int zeros = kStepK - min(kStepK, t.w - inner);  // in front of the window's last rows
                            tma_load_4d_pair(pb, &map_b, 0, -zeros, t.z + inner, n0 / 64, bar);
                            tma_load_4d_pair(pa, &map_a, 0, -zeros, t.z + inner, m0 / 64, bar);
                        } else {
                            if constexpr (kBMn)
                                tma_load_3d_pair(pb, &map_b, 0, p * pr.K + inner, n0 / 64, bar);
                            else
                                tma_load_2d_pair(pb, &map_b, inner, p * (OP == Op::kUp ? 2 : 1) * pr.N + n0, bar);
                            if (t.w == kHalfM) {
                                tma_load_2d_pair(pa, &map_a, inner, t.z, bar);
                            } else {
                                for (int i = 0; i < kHalfM / kRowBox; ++i)
                                    tma_load_2d_pair(pa + i * kBoxBytes, &map_a_small, inner, i < small ? t.z + i * kRowBox : pr.rows, bar);
                            }
                        }
                    } else {
                        uint64_t* bar = &b.full[s];
                        mbar_expect_tx(bar, bytes);
                        for (int i = 0; i < (two ? 2 : 1); ++i) {  // 128 columns each
                            if constexpr (kBMn)
                                tma_load_3d(pb + i * kGroup * kLine, &map_b, 0, p * pr.K + inner, n0 / 64 + 2 * i, bar);
                            else
                                tma_load_2d(pb + i * kGroup * kLine, &map_b, inner,
                                            p * (OP == Op::kUp ? 2 : 1) * pr.N + n0 + i * (OP == Op::kUp ? pr.N : kGroup), bar);
                        }
                        if (!few) {
                            tma_load_2d(pa, &map_a, inner, t.z, bar);
                        } else {
                            for (int i = 0; i < small; ++i)
                                tma_load_2d(pa + i * kBoxBytes, &map_a_small, inner, t.z + i * kRowBox, bar);
                        }
                    }
                    ++issued;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) set_error(pr.err, MOE_DEVERR_STALL);
            // Leave only after the copies in flight have landed and been read (or
            // never will), also where this thread was through before another wait gave up.
            const uint64_t t0 = now_ns();
            for (uint32_t i = issued > (uint32_t)stages ? issued - stages : 0; i < issued; ++i)
                while (!mbar_try(smem_u32(&b.empty[i % stages]), (i / stages) & 1) && now_ns() - t0 < kStallNs) {
                }
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0 && elect_one()) {
            bool ok = true;
            const uint64_t desc_a = kGrad ? umma_desc_mn(smem, kBlockBytes) : umma_desc(smem);
            const uint64_t desc_b = kBMn ? umma_desc_mn(smem + kABytes, kBlockBytes) : umma_desc(smem + kABytes);
            // From one 16 of the inner dimension to the next: 32 bytes along a row, or 16 rows.
            constexpr uint32_t kNextA = kGrad ? 16 * kLine / 16 : 2, kNextB = kBMn ? 16 * kLine / 16 : 2;
            const auto commit = [](uint64_t* bar) {
                if (PAIR)
                    umma_commit_pair(bar);
                else
                    umma_commit(bar);
            };
            int s = 0;
            uint32_t phase = 0, j = 0, unit = 0;  // tiles and chunks of this pair
            for (long long tile = pair; ok && tile < tiles; tile += pairs, ++j) {
                if (!(ok = tile_written(j))) break;
                const int4 t = tile_at(j);
                const bool two = OP == Op::kUp || 2 * t.y + 1 < blocks;
                const uint32_t idesc = umma_idesc_bf16(kTileM, two ? kTileN : kGroup, kGrad, kBMn);
                const int steps = steps_of(t);
                for (int k0 = 0; ok && k0 < steps; k0 += min(kChunk, steps - k0), ++unit) {
                    const uint32_t buf = unit & 1, d = tmem + buf * kTileN;
                    const int end = k0 + min(kChunk, steps - k0);
                    if (!(ok = mbar_wait_pair(&b.acc_empty[buf], ((unit >> 1) & 1) ^ 1, gave_up))) break;
                    for (int k = k0; k < end; ++k) {
                        // a pair's stage is written by both CTAs' copies
                        ok = PAIR ? mbar_wait_pair(&b.full[s], phase, gave_up) : mbar_wait(&b.full[s], phase, gave_up);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t da = desc_a + (uint32_t)s * (kStageBytes / 16);
                        const uint64_t db = desc_b + (uint32_t)s * (kStageBytes / 16);
                        // 16 rows in front of the window's last ones are left out (but one of an empty window's)
                        const int from = kGrad ? min(kStepK / 16 - 1, max(0, kStepK - (t.w - k * kStepK)) >> 4) : 0;
#pragma unroll
                        for (int i = 0; i < kStepK / 16; ++i)
                            if (i >= from) {
                                if (PAIR)
                                    umma_bf16_pair(d, da + i * kNextA, db + i * kNextB, idesc, k > k0 || i > from);
                                else
                                    umma_bf16(d, da + i * kNextA, db + i * kNextB, idesc, k > k0 || i > from);
                            }
                        commit(&b.empty[s]);
                        if (++s == stages) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok) commit(&b.acc_full[buf]);
                }
            }
            if (!ok) set_error(pr.err, MOE_DEVERR_STALL);
        }
    } else if (warp < kSumWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        // Finishing warps: warp w reads TMEM lanes 32 (w mod 4) .. + 31 (a row a
        // lane) and one half of the tile's columns.
        const int quarter = warp & 3, half = warp >> 2;
        const Boxes box = {staging + warp * kWarpBytes, lane};
        const uint32_t c0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * (OP == Op::kUp ? 64 : kGroup);
        const uint32_t c1 = c0 + (OP == Op::kUp ? kGroup : 64);
        const uint32_t acc_empty = PAIR ? peer_smem(smem_u32(&b.acc_empty[0]), 0) : smem_u32(&b.acc_empty[0]);
        uint32_t j = 0, unit = 0;
        // These warps run on after a wait has given up, so that up's pass the same
        // barriers in every tile: from the next tile on they have no rows and wait for
        // no sums (the results are void, and reported so).
        for (long long tile = pair; tile < tiles; tile += pairs, ++j) {
            const int4 t = __all_sync(kFull, tile_written(j)) ? tile_at(j) : make_int4(kGrad ? -1 : 0, 0, 0, 0);
            const int row = (kGrad ? t.x : t.z) + quarter * 32;
            const int rows = kGrad ? (t.x >= 0 ? kRowBox : 0) : max(0, min(kRowBox, t.w - quarter * 32));
            const int blk = 2 * t.y + half;  // this half's 128 columns (up: of another kind)
            const bool busy = rows > 0 && (OP == Op::kUp || blk < blocks);
            const int steps = __any_sync(kFull, *gave_up != 0) ? 0 : steps_of(t);
            Sums s;
            RowScalars rs;
            if (OP == Op::kDownBack && busy) rs = row_scalars(pr, (size_t)row + min(lane, rows - 1), blk);
            for (int k0 = 0; k0 < steps; k0 += min(kChunk, steps - k0), ++unit) {
                const uint32_t buf = unit & 1;
                mbar_pass(smem_u32(&b.acc_full[buf]), (unit >> 1) & 1, gave_up);
                tc_fence_after();
                if (busy) {
                    if (k0 == 0)
                        take_sums<true>(s, c0 + buf * kTileN, c1 + buf * kTileN);
                    else
                        take_sums<false>(s, c0 + buf * kTileN, c1 + buf * kTileN);
                }
                // the accumulator is read: it may be written again
                tc_fence_before();
                __syncwarp();
                if (elect_one()) {
                    if (PAIR)
                        mbar_signal_cluster(acc_empty + 8 * buf);
                    else
                        mbar_arrive(acc_empty + 8 * buf);
                }
            }
            if constexpr (OP == Op::kUp) {
                finish_up(pr, &map_out, &map_out2, box, staging + (warp ^ 4) * kWarpBytes, s, quarter, half, t.y, row,
                          rows);
                continue;
            }
            if (!busy) continue;
            if constexpr (OP == Op::kDownBack)
                finish_down_back(pr, &map_out, &map_out2, box, s, rs, blk, row, rows);
            else if constexpr (!kGrad)
                finish_rows(&map_out, box, s, blk * kGroup, row, rows, pr.out, pr.N);
            else if (pr.grad == MOE_GRAD_BF16)
                finish_rows(&map_out, box, s, blk * kGroup, row, rows, static_cast<uint16_t*>(pr.dw), pr.N);
            else if (pr.grad == MOE_GRAD_F32 || t.w > 0)
                finish_grad(&map_out, box, s, blk * kGroup, row, pr.grad == MOE_GRAD_F32_ADD);
        }
        if (elect_one()) bulk_wait();
        __syncwarp();
        if (*gave_up && lane == 0) set_error(pr.err, MOE_DEVERR_STALL);
        tc_fence_before();
    }
    // Neither CTA leaves while the other may still reach its shared memory or TMEM.
    // (A hardware barrier of threads whose waits have all ended.)
    __syncwarp();
    if (PAIR) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        if (PAIR)
            tmem_free_all_pair(tmem);
        else
            tmem_free_all(tmem);
    }
}

// ---- host side ----

constexpr CUtensorMapDataType kByte = CU_TENSOR_MAP_DATA_TYPE_UINT8, kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              kF32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;

template <Op OP, bool PAIR>
int launch_form(Problem pr, const uint16_t* a, const uint16_t* w, cudaStream_t s) {
    constexpr bool kGrad = OP == Op::kGrad;
    constexpr bool kBMn = OP == Op::kDownBack || OP == Op::kUpBack || kGrad;
    constexpr int kTileM = tile_m(PAIR);
    const int blocks = pr.N / kGroup, n_tiles = OP == Op::kUp ? blocks : (blocks + 1) / 2;
    // The most tiles any windows over these rows can have.
    const long long m_most = kGrad ? (long long)pr.P * ((pr.K + kTileM - 1) / kTileM)
                                   : ((long long)pr.rows + kTileM - 1) / kTileM + min(pr.P, pr.rows);
    if (m_most * n_tiles > INT32_MAX) return MOE_ERR_SIZE;
    const size_t rows = (size_t)pr.rows, n_rows = (size_t)pr.P * pr.N, k_rows = (size_t)pr.P * pr.K;
    CUtensorMap map_a, map_a_small, map_b, map_out, map_out2, map_codes;
    bool ok = kGrad ? window_map(&map_a, a, rows, pr.K, kStepK)
                    : tile_map(&map_a, kBf16, a, rows, pr.K, kHalfM) && tile_map(&map_a_small, kBf16, a, rows, pr.K, kRowBox);
    if (kGrad) map_a_small = map_a;
    ok = ok && (kGrad  ? window_map(&map_b, w, rows, pr.N, kStepK)
                : kBMn ? block_map(&map_b, w, k_rows, pr.N, kStepK)
                       : tile_map(&map_b, kBf16, w, (OP == Op::kUp ? 2 : 1) * n_rows, pr.K, kGroup));
    if (kGrad)
        ok = ok && tile_map(&map_out, pr.grad == MOE_GRAD_BF16 ? kBf16 : kF32, pr.dw, k_rows, pr.N, kRowBox);
    else
        ok = ok && tile_map(&map_out, kBf16, pr.out, rows, pr.N, kRowBox);
    map_out2 = map_out;
    if (OP == Op::kUp && pr.codes != nullptr) ok = ok && tile_map(&map_out2, kByte, pr.codes, rows, 2 * pr.N, kRowBox);
    map_codes = map_out2;
    if (OP == Op::kDownBack)
        ok = ok && tile_map(&map_out2, kBf16, pr.dgu, rows, 2 * pr.N, kRowBox) &&
             tile_map(&map_codes, kByte, pr.codes, rows, 2 * pr.N, kHalfM);
    if (!ok) return MOE_ERR_CUDA;
    // One stage less where the prefix of the windows leaves no room for it.
    constexpr int kStages = stages_of(OP, PAIR);
    pr.stages = kStages - (smem_bytes(OP, PAIR, kStages, pr.P) <= kSmemLimit ? 0 : 1);
    const auto kernel = dense_kernel<OP, PAIR>;
    // The same limit for every size, so that callers on several threads do not lower it for each other.
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess)
        return MOE_ERR_CUDA;
    constexpr int kCtas = PAIR ? 2 : 1;
    const int most = sm_count() / kCtas;
    if (most < 1) return MOE_ERR_CUDA;
    const unsigned grid = kCtas * (unsigned)(m_most * n_tiles < most ? m_most * n_tiles : most);
    const size_t smem = smem_bytes(OP, PAIR, pr.stages, pr.P);
    const dim3 block(kDenseThreads);
    const cudaError_t e = PAIR ? launch_pdl_cluster(0, 2, kernel, dim3(grid), block, smem, s, map_a, map_a_small, map_b,
                                                    map_out, map_out2, map_codes, pr)
                               : launch_pdl(kernel, dim3(grid), block, smem, s, map_a, map_a_small, map_b, map_out,
                                            map_out2, map_codes, pr);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Pairs, unless the average window fits a single CTA's rows: then the weights are the
// time, and single CTAs are faster.  Single CTAs / pairs: up of 1 token over 256
// experts of 7168 x 2048 80.1 / 86.8 us, down of 96 tokens 933 / 1000, up of 1024
// tokens over 64 such experts (128 rows each) 606 / 652; 1537 tokens over 44 experts
// of 1920 x 896 (175 rows each) up 68.5 / 67.5, up_back 71.3 / 67.4.  The rule knows
// the average alone (the windows are on the device).  Where the same rows fill a few
// long windows, pairs would be faster: 8192 rows over 64 experts of 7168 x 2048 (the
// rule's border) in all 64 windows, up 567 / 602; in 16 of them 310 / 274, in 2
// 300 / 261; of 2048 x 1024, 96 / 98, 57 / 50, 47 / 43.
template <Op OP>
int launch_dense(const Problem& pr, const uint16_t* a, const uint16_t* w, cudaStream_t s) {
    if constexpr (OP == Op::kUp || OP == Op::kDown || OP == Op::kUpBack)
        if ((long long)pr.rows <= (long long)pr.P * kHalfM) return launch_form<OP, false>(pr, a, w, s);
    return launch_form<OP, true>(pr, a, w, s);
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
    pr.P = e->P, pr.N = N, pr.K = M, pr.offsets = offsets, pr.rows = rows;
    pr.dw = dw, pr.grad = grad, pr.err = e->error_word;
    return launch_dense<Op::kGrad>(pr, a, b, s);
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
    pr.P = e->P, pr.N = e->I, pr.K = e->H, pr.offsets = offsets, pr.rows = rows, pr.out = h;
    pr.codes = codes, pr.scales = scales, pr.scale_stride = scale_stride, pr.err = e->error_word;
    return launch_dense<Op::kUp>(pr, x, e->w13, static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API int moe_dense_down(const moe_dense* e, const uint16_t* h, const int32_t* offsets, int32_t rows,
                                      uint16_t* out, void* stream) {
    int rc = check_dense(e, rows);
    if (rc != MOE_OK) return rc;
    const void* need[] = {e->w2, h, offsets, out};
    if ((rc = check_pointers(need, rows)) != MOE_OK || rows == 0) return rc;
    Problem pr = {};
    pr.P = e->P, pr.N = e->H, pr.K = e->I, pr.offsets = offsets, pr.rows = rows, pr.out = out;
    pr.err = e->error_word;
    return launch_dense<Op::kDown>(pr, h, e->w2, static_cast<cudaStream_t>(stream));
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
    pr.P = e->P, pr.N = e->I, pr.K = e->H, pr.offsets = offsets, pr.rows = rows;
    pr.out = hg, pr.dgu = dgu, pr.codes = const_cast<uint8_t*>(codes), pr.scales = const_cast<float*>(scales);
    pr.scale_stride = scale_stride, pr.row_gates = row_gates, pr.parts = gate_parts, pr.err = e->error_word;
    return launch_dense<Op::kDownBack>(pr, dout, e->w2, static_cast<cudaStream_t>(stream));
}

extern "C" MOE_API int moe_dense_up_backward(const moe_dense* e, const uint16_t* dgu, const int32_t* offsets,
                                             int32_t rows, uint16_t* dx, void* stream) {
    int rc = check_dense(e, rows);
    if (rc != MOE_OK) return rc;
    const void* need[] = {e->w13, dgu, offsets, dx};
    if ((rc = check_pointers(need, rows)) != MOE_OK || rows == 0) return rc;
    Problem pr = {};
    pr.P = e->P, pr.N = e->H, pr.K = 2 * e->I, pr.offsets = offsets, pr.rows = rows;
    pr.out = dx, pr.err = e->error_word;
    return launch_dense<Op::kUpBack>(pr, dgu, e->w13, static_cast<cudaStream_t>(stream));
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
