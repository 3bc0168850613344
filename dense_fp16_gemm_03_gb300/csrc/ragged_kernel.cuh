// Products whose second matrix depends on the row: grouped products by expert
// (forward and both gradients) and low-rank adapters beside a shared
// projection, as one persistent, warp-specialised sm_103a kernel.
//
// The matrix with the ragged extent sits on the N side of the tensor-core
// instruction and the weights on its M side ("P" and "Q" below): the
// instruction's N is chosen per tile in steps of 16 (one CTA) or 32 (CTA pair),
// so a group of 40 rows costs 48 or 64 columns and not a whole tile, and a group
// of one row streams its weights at the memory's rate.  Per mode, with w, x, dy
// as the caller passes them:
//
//   kNT      y[t, n]  = sum_k w[g][n, k] x[t, k]     P = w[g] rows n, Q = x rows t
//   kNN      dx[t, k] = sum_n w[g][n, k] dy[t, n]    P = w[g] columns k, Q = dy rows t
//   kTN      dw[g][n, k] = sum_t dy[t, n] x[t, k]    P = dy columns n, Q = x columns k
//   kLoraU   u[t, r]  = s sum_k a[i][r, k] x[t, k]   P = a[i] rows r, Q = x rows t, kept where ids[t] = i
//   kLoraY   y[t, n]  = sum_k w[n, k] x[t, k] + sum_r b[i][n, r] u[t, r]
//                                                    kNT with one group, then K blocks of b[i] against u with
//                                                    the rows of other adapters zeroed, one per adapter of the tile
//                                                    and 32 of its rank
//
// EPI adds to kNT a bias, an activation and a residual and keeps z, and to kNN the derivative of the activation (LinearParams);
// SUM sums kNN's columns besides.  What the epilogue reads comes in 32 x 32 pieces by the way that the results leave, the first
// while the product still runs.
//
// u is an fp32 sum that the tensor cores take again as an operand.  Rounded to the operands' type it would add to y's error
// nearly as much as y's own rounding, so it goes in two values, hi = round(u) and lo = round(u - hi), 16 bits in bf16 and 22
// in fp16, side by side in one K block: b's 32 columns against hi, and again against lo.  (8192 rows of 16 prompts,
// 8192 x 4096, rank 64, bf16: relative error 0.00204 and 341 us with one value, 0.00166 and 349 with two; 32-bit sums
// throughout have 0.00166.)
//
// Everything but kTN yields tiles with the output column on tensor-memory
// lanes and the row on columns; the epilogue transposes 32 x 32 pieces through
// shared memory and stores only rows of the tile's own group, so tiles may read
// past a group's end (what is computed for the rows there is thrown away) but
// never write there.
//
// Two shapes.  A single CTA with 128 x 64 tiles in an eight-stage ring, for few
// rows: bound by HBM (64 groups with 256 rows, 2048 x 4096: 149 us for 1.01 GB,
// 6.8 TB/s).  A CTA pair with 256 x 256 tiles in a six-stage ring, for many:
// bound by the tensor cores under the board's power limit (8192^3 in one group:
// 1601 TFLOP/s sustained, beside 1592 of the dense 256 x 256 kernel), and with
// groups of unlike size by what the narrower tiles load per multiply (32 groups
// of 16384 rows in all, 4096 x 4096: 312 us with 512 rows each, 339 uneven).
//
// Roles (one CTA or a CTA pair per tile):
//   warp 0      TMA producer into a ring of 128-byte-swizzled stages
//   warp 1      tensor memory and the MMA issuer (of the pair's first CTA; kLoraY: in the second, the relay)
//   warps 2..   epilogue, on one of two accumulators while the other fills: four
//               warps, or eight that share the columns of 256-row tiles (with
//               short contractions the tile's end is the longer part: 24 groups
//               of 16121 rows in all, 2024 x 136, 34 us with four, 26.2 with eight)
//               (a SUM epilogue: warps 4.., 2 and 3 only hold registers for them)
//   the last 4  helper, where the mode has one: kTN without maps zeroes the rows
//               past a group's end in its last K block (both operands: a zero
//               times an infinity of the next group would be NaN); kLoraY builds
//               the masked u operand, and for the same reason takes infinities and
//               NaN out of the adapter's b and has the epilogue write NaN for them
//               into that adapter's own rows alone.  A stage that the helper touches
//               arrives on its CTA's `tail` barrier and is released to the MMA by
//               the `fixed` barrier (kLoraY: from the second CTA by way of the relay).
//
// Group ends are read on the device (no host copy of them exists): every CTA
// turns the offsets into a table of tile counts in shared memory, where all
// roles look their tiles up.
//
// Walks: data-parallel (tile u on worker u mod workers), or with `sk` each
// worker takes an equal run of all K-block iterations.  A run that stops inside a
// tile publishes its fp32 partial for the worker that holds the tile's last K
// block.  Workers walk their run backwards, so they publish first and wait last,
// and only ever for lower-numbered workers, which start no later: launches that
// share the GPU cannot hold each other up.  Sums are added in a fixed order:
// results repeat bit for bit.  Every flag is clear at the launch's end, also after
// an abort, so a replay of a captured launch never finds one of the last.
// (Handing each next tile to the worker that comes for it first, by a counter,
// took 2% longer for the uneven groups above and 5% for one group of as many
// rows: the number's way through the roles costs more than the balance brings.)
//
// Every wait is bounded as in gemm_kernel.cuh: past `wait_limit` cycles the
// thread records an error code, raises the CTA's abort flag, and all roles
// leave, wait for copies in flight, free tensor memory and return.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>
#include <type_traits>

#include "linear_act.cuh"
#include "ragged_ptx.cuh"
#include "sched.cuh"

namespace gemm_f16 {

constexpr int kRagBlockK = 64;       // 16-bit elements per 128-byte swizzled row
constexpr int kRagRank = 32;         // columns of b in an adapter's K block, each against the two parts of u
constexpr int kRagBand = 8;          // N-side tiles walked together before the M side advances
constexpr int kRagMaxGroups = 1024;  // entries of the shared-memory group table
constexpr int kRagHelpers = 128;     // threads of the helper warps: one for each row of a stage's M side
constexpr int kRagMaxSmem = 232448;  // 227 KB opt-in dynamic shared memory per CTA

enum RaggedMode : int { kNT = 0, kNN = 1, kTN = 2, kLoraU = 3, kLoraY = 4 };

// Device error word codes (low byte, as in gemm_kernel.cuh); bits 8.. hold the CTA index.
enum : uint32_t {
    kRagErrEmpty = 1,
    kRagErrFull = 2,
    kRagErrAccEmpty = 3,
    kRagErrAccFull = 4,
    kRagErrDrain = 5,
    kRagErrPartial = 6,
    kRagErrRingDrain = 7,
    kRagErrFixed = 10,   // the helper did not finish a stage in time
    kRagErrTail = 11,    // a group's last K block, or an adapter's b, did not arrive in time
};

struct RaggedParams {
    CUtensorMap tm_p;     // M-side operand
    CUtensorMap tm_q[3];  // N-side operand: boxes of a stage's whole, half and quarter N side (kTN: the first, 64 columns)
    CUtensorMap tm_x;     // kTN: the output; kLoraY: the adapters' b
    // MN-major operands again, as (64 columns, row, column group, matrix) with boxes of two neighbouring groups of 64
    // rows each: one copy for a CTA's 128 columns where two took 0.35 us a K block instead of 0.22.  Whole groups
    // only: the columns from 64 * groups on, and single groups, come by tm_p and tm_q.
    CUtensorMap tm_p2, tm_q2;
    uint32_t p_groups, q_groups;
    const int32_t *offsets;  // [groups + 1] row offsets (kNT, kNN, kTN), or null: one group of all rows
    uint32_t groups;         // groups, or row tiles (kLoraU, kLoraY)
    uint32_t rows;           // rows t
    uint32_t pdim;           // extent on the M side
    uint32_t qdim;           // kTN: extent on the N side
    uint32_t kdim;           // contraction extent (not kTN)
    uint32_t k_blocks;       // ceil(kdim / 64)
    uint32_t tiles_p;        // tiles along the M side
    uint32_t tiles_q;        // kTN, kLoraY: tiles along the N side
    uint32_t per;            // kLoraU, kLoraY: rows of a row tile
    FastDiv by[kRagBand + 1];  // by[d] divides by d; by[0] by kRagBand * tiles_p
    uint32_t sk;             // 1: equal runs of K-block iterations; 2 (with an epilogue): of those of the last, partial wave
    uint32_t bf16;           // operand type: 0 fp16, 1 bf16
    uint32_t out32;          // kTN: 1 = fp32 output
    void *out;
    const int32_t *ids;      // kLoraU, kLoraY: adapter of each row
    const int32_t *counts;   // adapters present in each row tile
    const int32_t *list;     // their numbers, `per` slots a row tile
    const float *scale;      // per adapter, or null
    uint32_t adapters;       // ids outside [0, adapters) have none
    const float *delta;      // kNT: added to the rows that have an adapter, [rows, pdim]; only this comes from the
                             // previous kernel, so only the epilogue waits for it
    const void *u;           // kLoraY: u [rows, rank], a word each: hi in its low half, lo in its high half
    uint32_t rank;
    uint32_t rank_blocks;    // ceil(rank / 32)
    const CUtensorMap *maps; // kTN: for each group tm_p, tm_q[0], tm_p2, tm_q2 that end with the group's rows, or null
    uint32_t part_rows;      // kTN: not 0: groups are cut into parts of this many rows, which then are the `groups` of the
    uint32_t whole_groups;   // launch, each with a matrix of its own in `out`; and the number of whole ones
    float *partials;         // sk: one 128 x QCAP fp32 tile per CTA
    uint64_t *flags;         // sk: one per CTA, `stamp` while its partial waits to be added
    uint64_t stamp;          // (its high word is the same for all launches, so its complements are no other launch's stamp)
    uint32_t skip_fill;      // test hook: ring fill of CTA 0 left undone while the error word is clear (~0u: none)
    long long wait_limit;
    uint32_t *error_word;
};

// kNT and kNN with an epilogue: what it reads and writes besides `out`.
struct LinearParams : RaggedParams {
    const void *bias;      // kNT: [groups, pdim], or null
    const void *in;        // kNT: the residual, kNN: z, [rows, pdim], or null
    void *kept;            // kNT: z [rows, pdim], or null
    float *sums;           // SUM: sums of dx's columns over the rows of each N-side tile
    uint32_t act;
    uint32_t first, chain; // SUM: K blocks of a whole tile's first chain, and of all others
};

// SUM: an epilogue with the sums of dx's columns.  The tensor cores round every sum of 16 products toward zero, so a long
// contraction loses what grows with its length (relative 4.3e-6 at 4096, 1.0e-6 at 1024): nothing that 16 bits show, but all of it
// is in a sum over rows that is kept in 32.  So a contraction of more than kRagChain K blocks is cut into chains with an
// accumulator each, in turn, which the epilogue adds up in its registers, rounding to nearest, and puts back into tensor memory
// in the last one's place: 8.5e-7 at 4096 and 5.8e-7 at 1024, where sums in fp32 throughout have 6.4e-7 and 2.4e-7.  (Normal
// values.  Of one sign, where nothing cancels, what is cut off is all on one side: one chain of 13 blocks loses 4.6e-6 in fp16 and
// 7e-7 in bf16, contractions of 14 to 256 blocks 2.8e-6 to 5.3e-6 and 3e-7 to 9e-7.)  Beside one
// chain: 16384 rows, 4096 x 4096, 331 us and 313; 32 groups of 16384 rows in all, 1024 x 2048, 80 to 89 and 72 to 87.  (All pieces
// kept in registers to the tile's end, so that both accumulators are free: the code is unrolled and waits for its
// instructions, 338 and 104 us, and half as long again for contractions of 512.)
constexpr int kRagChain = 13;

template <int MODE, int CG, int QCAP, int STAGES, bool EPI = false, bool SUM = false>
struct RaggedCfg {
    static_assert(!EPI || MODE == kNT || MODE == kNN, "epilogue");
    static_assert(!SUM || (EPI && MODE == kNN), "column sums");
    using Params = std::conditional_t<EPI, LinearParams, RaggedParams>;
    static_assert(CG == 1 || CG == 2, "cta group");
    static constexpr bool kPMn = (MODE == kNN || MODE == kTN);  // M-side operand MN-major
    static constexpr bool kQMn = (MODE == kTN);                 // N-side operand MN-major
    static constexpr bool kHelper = (MODE == kTN || MODE == kLoraY);
    // (kTN: eight warps' boxes of 128 bytes a row do not fit; of 64 bytes, or shared by two warps, they took 8 and
    // 2% longer than four for 16384 rows, 32 groups, 4096 x 4096)
    static constexpr int kEpiSets = ((QCAP == 256 && MODE != kTN) || EPI) ? 2 : 1;
    static constexpr int kEpiWarps = 4 * kEpiSets;
    // SUM with 128 sums a thread: the epilogue's two warpgroups take registers over from the first (three warps to a quarter of an
    // SM have 168 each: 3 x 168 = 72 + 2 x 216).  Only they ever ask for more, and the first gives before it does anything else.
    static constexpr bool kRegs = SUM && QCAP == 256;
    static constexpr uint32_t kRegsFirst = 72, kRegsEpi = 216, kRegsAll = 168;
    static constexpr int kFirstEpi = kRegs ? 4 : 2;             // warp
    static constexpr int kFirstHelper = kFirstEpi + kEpiWarps;  // warp
    static constexpr int kThreads = 32 * kFirstHelper + (kHelper ? kRagHelpers : 0);
    static constexpr int kQCta = QCAP / CG;                     // N-side extent in one CTA's stage
    // rows of a whole N-side box; a tile takes at most two boxes (halves and quarters) and at most a quarter's
    // rows too many, because every further box in a K block costs the producer more than the rows do
    static constexpr int kQBox = kQCta;
    static constexpr int kPBytes = 128 * 128;
    static constexpr int kQBytes = kQCta * 128;
    static constexpr int kStep = 16 * CG;                       // granularity of the instruction's N
    static constexpr int kOffP = 0;
    static constexpr int kOffQ = STAGES * kPBytes;
    static constexpr int kOffStore = kOffQ + STAGES * kQBytes;  // per epilogue warp
    static constexpr int kStoreBytes = (MODE == kTN) ? 4096 : 2048;
    static constexpr int kOffTabRow = kOffStore + kEpiWarps * kStoreBytes;
    static constexpr int kOffTabTile = kOffTabRow + 4 * (kRagMaxGroups + 4);
    // full, empty, fixed, tail per stage; acc_full x2, acc_empty x2, drain, bad_free x2
    static constexpr int kNumBars = 4 * STAGES + 7;
    // kLoraY: for each of two tiles in flight, 128 bits per adapter of the tile (b rows that hold an infinity or
    // NaN), and for each helper warp whether it found any
    static constexpr int kOffBad = kOffTabTile + 4 * (kRagMaxGroups + 4);
    static constexpr int kBadBytes = (MODE == kLoraY) ? QCAP * 16 : 0;
    static constexpr int kOffBar = kOffBad + 2 * kBadBytes;
    // last fill of each stage: its number + 1, this CTA's bytes, the bytes armed, 1 if it went to the tail barrier
    static constexpr int kOffRec = kOffBar + kNumBars * 8;
    static constexpr int kOffTmemSlot = kOffRec + STAGES * 16;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr int kOffAnyBad = kOffAbort + 4;
    // column sums on their way from the second epilogue set to the first, of two tiles
    static constexpr int kOffSums = kOffAnyBad + 32;
    static constexpr int kSmemBytes = kOffSums + (SUM ? 2 * 128 * 4 : 0) + 1024;
    static constexpr int kTmemCols = 2 * QCAP < 32 ? 32 : 2 * QCAP;
    static_assert(kQBytes % 1024 == 0 && kOffBar % 8 == 0, "layout");
    static_assert(kSmemBytes <= kRagMaxSmem, "shared memory budget");
    static_assert(QCAP % (32 * CG) == 0 && QCAP <= 256, "N side");
    static_assert(!kQMn || kQCta % 64 == 0, "whole 64-column atoms");
};

// One run of K blocks [lo, hi) of a tile.
struct RaggedSeg {
    uint32_t tile;
    uint32_t g;       // group (kNT, kNN, kTN), row tile (kLoraU, kLoraY)
    uint32_t p0;      // M-side origin of the tile (of the pair)
    uint32_t q0;      // first row (kTN: column) on the N side
    uint32_t qi;      // kNT, kNN: number of the tile among those of the group's rows
    uint32_t qn;      // rows (columns) of the tile that count
    uint32_t nq;      // the instruction's N
    uint32_t row0;    // kTN: first row of the group; kLoraU: the adapter
    uint32_t krows;   // kTN: rows of the group
    uint32_t kb;      // K blocks of the whole tile
    uint32_t lo, hi;
    uint32_t slots;   // kLoraY: adapters of the tile
    uint32_t extra;   // kLoraY: how many of the K blocks are theirs
    uint32_t e_lo, e_hi;  // and which of those lie in [lo, hi)
};

// The order of a kLoraY tile's K blocks: items, the projection's blocks and the adapters, each adapter's blocks in a row.  The
// adapters are spread evenly between the others, so that the helper prepares one while the tensor cores work on the others,
// and every run of a split tile has its share.  An adapter's blocks come later than the ring can look ahead, by some 1.6 us
// (their load, the helper, the release to the pair's first CTA), but the blocks of one adapter share that: 2048 rows with
// one of 64 adapters of rank 64 each, 4096 x 4096, took 620 us with the blocks spread one by one, 529 in a row and released
// two at a time, and 413 with the relay.  Item i is an adapter where floor(i slots / items) steps.
struct RaggedMix {
    uint32_t items, slots, blocks, left, run, begun, e, m;  // left = i slots mod items; run: blocks of the present adapter
                                                            // still to come; adapters begun, adapter and projection blocks
    __device__ __forceinline__ RaggedMix(const RaggedSeg &s, uint32_t rank_blocks) : slots(s.slots), blocks(rank_blocks)
    {
        items = s.kb - s.extra + s.slots;
        e = s.e_lo;
        m = s.lo - e;
        left = run = begun = 0u;
        if (e != 0u) {
            const uint32_t j = (e + blocks - 1u) / blocks;
            run = j * blocks - e;
            begun = j;
            left = uint32_t(uint64_t(m + j) * slots - uint64_t(j) * items);
        } else {
            left = m * slots;
        }
    }
    // whether the current block is an adapter block; then on to the next
    __device__ __forceinline__ bool step()
    {
        if (run != 0u) {
            --run;
            ++e;
            return true;
        }
        left += slots;
        if (left >= items) {
            left -= items;
            run = blocks - 1u;
            ++begun;
            ++e;
            return true;
        }
        ++m;
        return false;
    }
    // adapter blocks before block v
    static __device__ __forceinline__ uint32_t before(const RaggedSeg &s, uint32_t v, uint32_t blocks)
    {
        if (v == 0u || s.extra == 0u) return 0u;
        if (v == s.kb) return s.extra;
        const uint32_t items = s.kb - s.extra + s.slots;
        uint32_t i = v;
        if (blocks > 1u) {  // the last item that begins at v or before
            uint32_t lo = 0u, hi = min(v, items - 1u);
            while (lo < hi) {
                const uint32_t mid = (lo + hi + 1u) >> 1;
                if (mid + (blocks - 1u) * uint32_t(uint64_t(mid) * s.slots / items) <= v) lo = mid;
                else hi = mid - 1u;
            }
            i = lo;
        }
        const uint32_t j = uint32_t(uint64_t(i) * s.slots / items);
        return j * blocks + (v - i - j * (blocks - 1u));
    }
};

// The adapters of a kLoraY tile by slot, 32 at a time in the lanes of a warp: the list's latency is not on the way of every
// block.  Called by whole warps.
struct RaggedNames {
    const int32_t *list;
    uint32_t slots, chunk;
    int32_t name;
    __device__ __forceinline__ RaggedNames(const int32_t *of_tile, uint32_t count, uint32_t slot) : list(of_tile), slots(count)
    {
        load(slot >> 5);
    }
    __device__ __forceinline__ void load(uint32_t c)
    {
        chunk = c;
        const uint32_t i = 32u * c + (threadIdx.x & 31u);
        name = i < slots ? list[i] : -1;
    }
    __device__ __forceinline__ int32_t operator[](uint32_t slot)
    {
        if ((slot >> 5) != chunk) load(slot >> 5);
        return __shfl_sync(0xffffffffu, name, slot & 31u);
    }
};

template <int CG>
__device__ __forceinline__ bool ragged_wait(uint32_t bar, uint32_t parity, const RaggedParams &p,
                                            volatile uint32_t *abort_flag, uint32_t code)
{
    auto try_once = [&]() {
        if constexpr (CG > 1) return ptx::mbar_try_wait_cluster(bar, parity);
        else return ptx::mbar_try_wait(bar, parity);
    };
    if (try_once()) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (try_once()) return true;
        if ((it & 31u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > p.wait_limit) {
                *abort_flag = 1u;
                atomicCAS(p.error_word, 0u, code | (blockIdx.x << 8));
                return false;
            }
        }
    }
}

// The same wait by a whole warp, which leaves it together.
template <int CG>
__device__ __forceinline__ bool ragged_wait_warp(uint32_t bar, uint32_t parity, const RaggedParams &p,
                                                 volatile uint32_t *abort_flag, uint32_t code)
{
    const bool ok = ragged_wait<CG>(bar, parity, p, abort_flag, code);
    return __all_sync(0xffffffffu, ok);
}

// A value all lanes hold, in a form the compiler can keep in uniform registers: the operands of TMA and MMA
// instructions live there, and moving them over for every instruction delays the issue loops.
__device__ __forceinline__ uint32_t uniform(uint32_t v)
{
    return __reduce_or_sync(0xffffffffu, v);
}

template <int MODE>
__device__ __forceinline__ void uniform(RaggedSeg &s)
{
    s.g = uniform(s.g);
    s.p0 = uniform(s.p0);
    s.q0 = uniform(s.q0);
    s.nq = uniform(s.nq);
    s.lo = uniform(s.lo);
    s.hi = uniform(s.hi);
    s.kb = uniform(s.kb);
    if constexpr (MODE == kTN || MODE == kLoraU) s.row0 = uniform(s.row0);
    if constexpr (MODE == kTN) s.krows = uniform(s.krows);
    if constexpr (MODE == kLoraY) {
        s.slots = uniform(s.slots);
        s.extra = uniform(s.extra);
        s.e_lo = uniform(s.e_lo);
        s.e_hi = uniform(s.e_hi);
    }
}

// The flag of a partial sum.  A launch captured in a graph comes again with the same stamp, so whatever happens in a launch,
// its end finds the flag cleared: of the CTA that has the sum to publish and the one that takes it, each writes the flag
// once, also where it gives up, and the one that comes second clears it.
__device__ __forceinline__ uint64_t flag_given_up(uint64_t stamp)  // by the taker
{
    return ~stamp;
}

__device__ __forceinline__ uint64_t flag_not_coming(uint64_t stamp)  // by the publisher
{
    return stamp ^ (uint64_t(1) << 63);
}

// `v`: the stamp, or flag_not_coming.
__device__ __forceinline__ void flag_publish(uint64_t *flag, uint64_t stamp, uint64_t v)
{
    if (ptx::exch_gpu_u64(flag, v) == flag_given_up(stamp)) ptx::st_release_gpu_u64(flag, 0u);
}

__device__ __forceinline__ void flag_give_up(uint64_t *flag, uint64_t stamp)
{
    const uint64_t old = ptx::exch_gpu_u64(flag, flag_given_up(stamp));
    if (old == stamp || old == flag_not_coming(stamp)) ptx::st_release_gpu_u64(flag, 0u);
}

template <int MODE, int CG, int QCAP, bool EPI>
struct RaggedWalk {
    const RaggedParams &p;
    const int32_t *tab_row;    // offsets (groups + 1), or counts per row tile
    const uint32_t *tab_tile;  // tiles before each group (groups + 1)
    const int32_t *list;       // kLoraU, kLoraY: the adapters of each row tile
    uint32_t worker, workers, total;
    uint32_t run, longer;      // sk: K-block iterations of a worker; the first `longer` workers have one more
    uint32_t tile_blocks;      // sk: K blocks of every tile
    uint32_t splitters, whole; // sk 2: workers that have a run, and tiles before the split ones

    // A producer that is late with a tile's first load leaves the ring short for the rest of it, so the way from a tile's
    // number to its place is kept short: the group is looked for from the last one on, and divisors are known.  `near` is
    // the group of the tile before (any group at first).
    __device__ __forceinline__ void decode(uint32_t u, RaggedSeg &s, uint32_t &near) const
    {
        constexpr uint32_t kStep = 16u * CG;
        s.tile = u;
        if constexpr (MODE == kLoraY) {
            uint32_t pi, qi;
            raster(u, p.tiles_q, pi, qi);
            s.g = qi;
            s.p0 = pi * 128u * CG;
            s.q0 = qi * p.per;
            s.qn = min(p.per, p.rows - s.q0);
            s.row0 = 0;
            s.slots = uint32_t(tab_row[qi]);
            s.extra = s.slots * p.rank_blocks;
            s.kb = p.k_blocks + s.extra;
        } else {
            uint32_t lo = near;  // the group with tab_tile[lo] <= u < tab_tile[lo + 1]
            for (int i = 0; i < 3 && tab_tile[lo + 1] <= u; ++i) ++lo;
            if (tab_tile[lo] > u || tab_tile[lo + 1] <= u) {
                lo = 0;
                uint32_t hi = p.groups;
                while (hi - lo > 1u) {
                    const uint32_t mid = (lo + hi) >> 1;
                    if (tab_tile[mid] <= u) lo = mid;
                    else hi = mid;
                }
            }
            near = lo;
            s.g = lo;
            const uint32_t local = u - tab_tile[lo];
            s.kb = p.k_blocks;
            if constexpr (MODE == kLoraU) {
                s.p0 = 0;
                s.q0 = lo * p.per;
                s.qn = min(p.per, p.rows - s.q0);
                s.row0 = uint32_t(list[size_t(lo) * p.per + local]);
            } else {
                const uint32_t r0 = uint32_t(tab_row[lo]);
                const uint32_t rows = uint32_t(tab_row[lo + 1]) - r0;
                uint32_t pi, qi;
                if constexpr (MODE == kTN) {
                    raster(local, p.tiles_q, pi, qi);
                    s.q0 = qi * QCAP;
                    s.qn = min(uint32_t(QCAP), p.qdim - s.q0);
                    s.row0 = r0;
                    s.krows = rows;
                    s.kb = (rows + kRagBlockK - 1u) / kRagBlockK;
                } else {
                    // equal tiles, in whole steps of the instruction's N (one tile: no division on the way to the
                    // first load)
                    pi = local;
                    qi = 0u;
                    s.q0 = r0;
                    s.qn = rows;
                    if (rows > uint32_t(QCAP)) {
                        const uint32_t tq = (rows + QCAP - 1u) / QCAP;
                        const uint32_t share = tq <= uint32_t(kRagBand) ? fast_div(p.by[tq], rows + tq - 1u) : (rows + tq - 1u) / tq;
                        const uint32_t each = (share + kStep - 1u) / kStep * kStep;
                        raster(local, tq, pi, qi);
                        s.q0 = r0 + qi * each;
                        s.qn = min(each, r0 + rows - s.q0);
                    }
                    s.row0 = r0;
                    s.qi = qi;
                }
                s.p0 = pi * 128u * CG;
            }
        }
        s.nq = (s.qn + kStep - 1u) / kStep * kStep;
    }

    // tile `t` of a tiles_p x tq grid, walked in bands of N-side tiles, N side fastest
    __device__ __forceinline__ void raster(uint32_t t, uint32_t tq, uint32_t &pi, uint32_t &qi) const
    {
        uint32_t b = 0, w = tq;
        if (tq > uint32_t(kRagBand)) {
            b = fast_div(p.by[0], t);
            t -= b * p.by[0].d;
            w = min(uint32_t(kRagBand), tq - b * kRagBand);
        }
        pi = fast_div(p.by[w], t);
        qi = b * kRagBand + (t - pi * w);
    }

    __device__ __forceinline__ void count_extra(RaggedSeg &s) const
    {
        if constexpr (MODE == kLoraY) {
            s.e_lo = RaggedMix::before(s, s.lo, p.rank_blocks);
            s.e_hi = RaggedMix::before(s, s.hi, p.rank_blocks);
        } else {
            s.e_lo = s.e_hi = 0u;
        }
    }

    // sk: all tiles have the same K blocks (kLoraY: there is one row tile).  A run shorter than kMinRun blocks
    // would cost more in adding partials than it saves, so few iterations go to fewer workers.
    static constexpr uint32_t kMinRun = 4;
    __device__ __forceinline__ void plan_runs()
    {
        if (MODE == kTN || !p.sk || total == 0u) return;
        tile_blocks = p.k_blocks;
        if (MODE == kLoraY) tile_blocks += uniform(uint32_t(tab_row[0])) * p.rank_blocks;
        if constexpr (EPI) {
            // sk 2: the tiles that fill no wave are split, the others follow whole
            splitters = workers;
            whole = p.sk == 2u ? total / workers * workers : 0u;
            const uint32_t iters = (total - whole) * tile_blocks;
            splitters = min(workers, max(1u, iters / kMinRun));
            run = iters / splitters;
            longer = iters - run * splitters;
            return;
        }
        const uint32_t iters = total * tile_blocks;  // below 2^32: the host checks
        const uint32_t most = max(1u, iters / kMinRun);
        if (most < workers) workers = most;
        run = iters / workers;
        longer = iters - run * workers;
    }
    __device__ __forceinline__ uint32_t first_split() const  // tile
    {
        return EPI ? whole : 0u;
    }
    __device__ __forceinline__ uint32_t run_begin(uint32_t w) const
    {
        return w * run + min(w, longer);
    }

    // the first of the workers before this one that hold K blocks of the tile that starts at iteration `start`
    __device__ __forceinline__ uint32_t first_of(uint32_t start) const
    {
        uint32_t w = worker;
        while (w > 0u && run_begin(w) > start) --w;
        return w;
    }

    // sk, run by one warp of a CTA that stops early: what it has neither published nor taken, and now never will
    __device__ __forceinline__ void leave_flags(uint32_t rank, bool published, bool taken) const
    {
        const uint32_t lane = threadIdx.x & 31u, kb = tile_blocks;
        if (EPI && worker >= splitters) return;
        const uint32_t begin = run_begin(worker), end = run_begin(worker + 1u);
        const uint32_t start = begin / kb * kb;
        if (!published && lane == 0 && end % kb != 0u)  // the run stops inside a tile
            flag_publish(p.flags + worker * CG + rank, p.stamp, flag_not_coming(p.stamp));
        if (!taken && begin != start && end - start >= kb)  // it holds the end, not the beginning of its lowest tile
            for (uint32_t w = first_of(start) + lane; w < worker; w += 32u) flag_give_up(p.flags + w * CG + rank, p.stamp);
    }

    // f(seg) returns false to stop early (abort)
    template <bool UNIFORM, class F>
    __device__ __forceinline__ void each(F &&f) const
    {
        RaggedSeg s;
        uint32_t near = 0;
        if (MODE == kTN || !p.sk) {
            for (uint32_t u = worker; u < total; u += workers) {
                decode(u, s, near);
                s.lo = 0;
                s.hi = s.kb;
                count_extra(s);
                if constexpr (UNIFORM) uniform<MODE>(s);
                if (!f(s)) return;
            }
            return;
        }
        if (total == 0u || (!EPI && worker >= workers)) return;
        const uint32_t begin = EPI && worker >= splitters ? 0u : run_begin(worker);
        uint32_t it = EPI && worker >= splitters ? 0u : run_begin(worker + 1u);
        const uint32_t kb = tile_blocks;
        while (it > begin) {
            const uint32_t u = (it - 1u) / kb;
            const uint32_t start = u * kb;
            decode(first_split() + u, s, near);
            s.lo = begin > start ? begin - start : 0u;
            s.hi = it - start;
            const uint32_t lo = s.lo;
            count_extra(s);
            if constexpr (UNIFORM) uniform<MODE>(s);
            if (!f(s)) return;
            it = start + lo;
        }
        if constexpr (EPI) {
            for (uint32_t u = worker; u < whole; u += workers) {
                decode(u, s, near);
                s.lo = 0;
                s.hi = s.kb;
                count_extra(s);
                if constexpr (UNIFORM) uniform<MODE>(s);
                if (!f(s)) return;
            }
        }
    }
};

__device__ __forceinline__ uint32_t ragged_pack(float lo, float hi, bool bf16)
{
    if (bf16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

__device__ __forceinline__ float2 ragged_unpack(uint32_t w, bool bf16)
{
    if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// What is left of v beside its rounding `hi`: nothing where that is infinite or NaN.
__device__ __forceinline__ float ragged_rest(float v, float hi)
{
    return hi - hi == 0.0f ? v - hi : 0.0f;
}

// The group table: row offsets clamped to [0, rows] and made monotone (offsets that are not can
// then reach no other memory), and the number of tiles before each group.  Run by the whole CTA.
template <int MODE, int QCAP>
__device__ __forceinline__ void ragged_table(const RaggedParams &p, int32_t *tab_row, uint32_t *tab_tile)
{
    constexpr bool kOffsets = (MODE == kNT || MODE == kNN || MODE == kTN);
    const uint32_t n = (MODE == kTN && p.part_rows ? p.whole_groups : p.groups) + (kOffsets ? 1u : 0u);
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) {
        int32_t v;
        if (!kOffsets) v = p.counts[i];
        else if (p.offsets == nullptr) v = i ? int32_t(p.rows) : 0;  // one group of all rows
        else v = max(0, min(p.offsets[i], int32_t(p.rows)));
        tab_row[i] = v;
    }
    __syncthreads();
    if (threadIdx.x < 32u && MODE != kLoraY) {
        const uint32_t lane = threadIdx.x;
        if constexpr (kOffsets) {
            const uint32_t c = (n + 31u) / 32u, b = min(lane * c, n), e = min(b + c, n);
            int32_t top = 0;
            for (uint32_t i = b; i < e; ++i) top = max(top, tab_row[i]);
            int32_t before = top;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, before, d);
                if (lane >= uint32_t(d)) before = max(before, o);
            }
            before = __shfl_up_sync(0xffffffffu, before, 1);
            if (lane == 0) before = 0;
            for (uint32_t i = b; i < e; ++i) {
                before = max(before, tab_row[i]);
                tab_row[i] = before;
            }
            __syncwarp();
        }
    }
    if constexpr (MODE == kTN) {
        if (p.part_rows) {  // the table of the parts; those that there are not have no rows
            __syncthreads();
            const uint32_t i = threadIdx.x;
            const bool group = i + 1u < n;
            const int32_t begin = group ? tab_row[i] : 0, end = tab_row[n - 1u];
            const uint32_t count = group ? (uint32_t(tab_row[i + 1u] - begin) + p.part_rows - 1u) / p.part_rows : 0u;
            if (group) tab_tile[i] = count;
            __syncthreads();
            uint32_t first = 0, all = 0;
            for (uint32_t j = 0; j + 1u < n; ++j) {
                if (j == i) first = all;
                all += tab_tile[j];
            }
            __syncthreads();
            for (uint32_t j = 0; j < count; ++j) tab_row[first + j] = begin + int32_t(j * p.part_rows);
            for (uint32_t j = all + i; j <= p.groups; j += blockDim.x) tab_row[j] = end;
            __syncthreads();
        }
    }
    if (threadIdx.x < 32u && MODE != kLoraY) {
        const uint32_t lane = threadIdx.x;
        auto tiles = [&](uint32_t g) -> uint32_t {
            if constexpr (MODE == kLoraU) return uint32_t(tab_row[g]);
            const uint32_t rows = uint32_t(tab_row[g + 1] - tab_row[g]);
            if constexpr (MODE == kTN) return rows ? p.tiles_p * p.tiles_q : 0u;
            else return (rows + QCAP - 1u) / QCAP * p.tiles_p;
        };
        const uint32_t c = (p.groups + 31u) / 32u, b = min(lane * c, p.groups), e = min(b + c, p.groups);
        uint32_t sum = 0;
        for (uint32_t i = b; i < e; ++i) sum += tiles(i);
        uint32_t before = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= uint32_t(d)) before += o;
        }
        before -= sum;
        for (uint32_t i = b; i < e; ++i) {
            tab_tile[i] = before;
            before += tiles(i);
        }
        if (lane == 31u) tab_tile[p.groups] = before;
    }
    __syncthreads();
}

__device__ __forceinline__ float ragged_value(uint16_t v, bool bf16)
{
    return ragged_unpack(v, bf16).x;
}

// A piece of 32 rows x 32 columns of a row-major matrix, as an epilogue warp moves it: a lane has four neighbouring columns
// (8 bytes) of eight rows, a quarter of the warp 64 bytes of a row.  Between that and a column per lane lies a turn through
// the warp's buffer, 16 lines of 32 words: word l of line i holds rows 2i (low half) and 2i + 1 of column l.
template <bool USED>
struct LinearPiece {
    uint2 v[8];  // rows 2 (4i + lane / 8) + h in v[2i + h]
    __device__ __forceinline__ void fetch(const void *from, uint32_t pitch, const RaggedSeg &s, uint32_t prow, uint32_t c)
    {
        const uint32_t lane = threadIdx.x & 31u, col = prow + 4u * (lane & 7u);
        const char *at = static_cast<const char *>(from) + (size_t(s.q0) * pitch + col) * 2u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t row = 32u * c + 2u * (4u * uint32_t(i >> 1) + (lane >> 3)) + uint32_t(i & 1);
            v[i] = (col < pitch && row < s.qn) ? *reinterpret_cast<const uint2 *>(at + size_t(row) * pitch * 2u) : make_uint2(0u, 0u);
        }
    }
    // rows 2i and 2i + 1 of this lane's column in w[i]
    __device__ __forceinline__ void columns(uint32_t buf, uint32_t (&w)[16]) const
    {
        const uint32_t lane = threadIdx.x & 31u;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 a = v[2 * i], b = v[2 * i + 1];
            ptx::st_shared_v4(buf + (uint32_t(i) * 4u + (lane >> 3)) * 128u + (lane & 7u) * 16u, __byte_perm(a.x, b.x, 0x5410u),
                              __byte_perm(a.x, b.x, 0x7632u), __byte_perm(a.y, b.y, 0x5410u), __byte_perm(a.y, b.y, 0x7632u));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = ptx::ld_shared_u32(buf + uint32_t(i) * 128u + lane * 4u);
    }
};

template <>
struct LinearPiece<false> {
};

// The same piece the other way: 32 rows of this lane's column in fp32, rounded.
__device__ __forceinline__ void linear_store(void *to, uint32_t pitch, const RaggedSeg &s, uint32_t prow, uint32_t c, uint32_t buf,
                                             const uint32_t (&r)[32], bool bf16)
{
    const uint32_t lane = threadIdx.x & 31u, col = prow + 4u * (lane & 7u);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        ptx::st_shared_u32(buf + uint32_t(i) * 128u + lane * 4u,
                           ragged_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), bf16));
    __syncwarp();
    char *at = static_cast<char *>(to) + (size_t(s.q0) * pitch + col) * 2u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pr = uint32_t(i) * 4u + (lane >> 3);
        const uint4 v = ptx::ld_shared_v4(buf + pr * 128u + (lane & 7u) * 16u);
        const uint32_t row = 32u * c + 2u * pr;
        if (col >= pitch) continue;
        if (row < s.qn)
            ptx::st_global_v2(at + size_t(row) * pitch * 2u, __byte_perm(v.x, v.y, 0x5410u), __byte_perm(v.z, v.w, 0x5410u));
        if (row + 1u < s.qn)
            ptx::st_global_v2(at + size_t(row + 1u) * pitch * 2u, __byte_perm(v.x, v.y, 0x7632u), __byte_perm(v.z, v.w, 0x7632u));
    }
}

// After an abort: wait (bounded) until no copy into this CTA's ring, or armed on its barriers, is in
// flight.  Run by one thread of each CTA between the teardown's two cluster barriers; `own` and
// `peer` point at the two CTAs' fill records (peer 0: none).  The pair's first CTA owns the full
// barriers; a tail fill lands on its own CTA's tail barrier.
template <int STAGES, int CG>
__device__ __noinline__ void ragged_drain(uint32_t bars, uint32_t rec, bool leader, const RaggedParams &p)
{
    auto wait = [&](uint32_t bar, uint32_t parity) {
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(bar, parity)) {
            if (clock64() - t0 > p.wait_limit) {
                atomicCAS(p.error_word, 0u, kRagErrRingDrain | (blockIdx.x << 8));
                break;
            }
        }
    };
    for (uint32_t s = 0; s < uint32_t(STAGES); ++s) {
        const uint32_t a = rec + 16u * s;
        const uint32_t mine = ptx::ld_shared_cluster_u32(ptx::map_to_rank(a, ptx::cluster_ctarank()));
        const uint32_t own_rank = ptx::cluster_ctarank();
        const uint32_t my_bytes = ptx::ld_shared_cluster_u32(ptx::map_to_rank(a + 4u, own_rank));
        const uint32_t my_armed = ptx::ld_shared_cluster_u32(ptx::map_to_rank(a + 8u, own_rank));
        const uint32_t my_tail = ptx::ld_shared_cluster_u32(ptx::map_to_rank(a + 12u, own_rank));
        if (mine && (my_tail & 1u)) wait(bars + 8u * (3u * STAGES + s), my_tail >> 1);
        if (!leader) continue;
        uint32_t other = 0, other_bytes = 0, other_tail = 0;
        if constexpr (CG == 2) {
            other = ptx::ld_shared_cluster_u32(ptx::map_to_rank(a, 1u));
            other_bytes = ptx::ld_shared_cluster_u32(ptx::map_to_rank(a + 4u, 1u));
            other_tail = ptx::ld_shared_cluster_u32(ptx::map_to_rank(a + 12u, 1u));
        }
        const uint32_t bar = bars + 8u * s;
        if (mine >= other) {
            if (!mine || (my_tail & 1u)) continue;
            const uint32_t landing = my_bytes + (other == mine ? other_bytes : 0u);
            if (my_armed > landing) ptx::mbar_complete_tx(bar, my_armed - landing);
            wait(bar, ((mine - 1u) / STAGES) & 1u);
        } else if (!(other_tail & 1u)) {
            ptx::mbar_arrive_expect_tx(bar, other_bytes);
            wait(bar, ((other - 1u) / STAGES) & 1u);
        }
    }
}

__device__ __forceinline__ uint32_t ragged_first_chain(const LinearParams &p, const RaggedSeg &s)
{
    return s.lo == 0u && s.hi == s.kb ? p.first : p.chain;
}

template <int MODE, int CG, int QCAP, int STAGES, bool EPI = false, bool SUM = false>
__global__ void __launch_bounds__(RaggedCfg<MODE, CG, QCAP, STAGES, EPI, SUM>::kThreads, 1)
    gemm_ragged_kernel(const __grid_constant__ typename RaggedCfg<MODE, CG, QCAP, STAGES, EPI, SUM>::Params p)
{
    using Cfg = RaggedCfg<MODE, CG, QCAP, STAGES, EPI, SUM>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);

    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t rank = (CG == 2) ? ptx::cluster_ctarank() : 0u;
    const bool leader = (rank == 0);

    auto bar_full = [&](uint32_t s) { return base + Cfg::kOffBar + 8u * s; };
    auto bar_empty = [&](uint32_t s) { return base + Cfg::kOffBar + 8u * (STAGES + s); };
    auto bar_fixed = [&](uint32_t s) { return base + Cfg::kOffBar + 8u * (2 * STAGES + s); };
    auto bar_tail = [&](uint32_t s) { return base + Cfg::kOffBar + 8u * (3 * STAGES + s); };
    auto bar_acc_full = [&](uint32_t b) { return base + Cfg::kOffBar + 8u * (4 * STAGES + b); };
    auto bar_acc_empty = [&](uint32_t b) { return base + Cfg::kOffBar + 8u * (4 * STAGES + 2 + b); };
    const uint32_t bar_drain = base + Cfg::kOffBar + 8u * (4 * STAGES + 4);
    auto bar_bad_free = [&](uint32_t b) { return base + Cfg::kOffBar + 8u * (4 * STAGES + 5 + b); };
    volatile uint32_t *any_bad = reinterpret_cast<volatile uint32_t *>(smem + Cfg::kOffAnyBad);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + Cfg::kOffAbort);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::kOffTmemSlot);
    volatile uint32_t *rec = reinterpret_cast<volatile uint32_t *>(smem + Cfg::kOffRec);
    int32_t *tab_row = reinterpret_cast<int32_t *>(smem + Cfg::kOffTabRow);
    uint32_t *tab_tile = reinterpret_cast<uint32_t *>(smem + Cfg::kOffTabTile);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(bar_full(s), 1);
            ptx::mbar_init(bar_empty(s), 1);
            // (kLoraY: each CTA's own helpers, and in the pair's first CTA the other's relay)
            ptx::mbar_init(bar_fixed(s), MODE == kLoraY ? kRagHelpers / 32 + (leader ? 1 : 0) : (kRagHelpers / 32) * CG);
            ptx::mbar_init(bar_tail(s), 1);
            rec[4 * s] = 0u;
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar_acc_full(b), 1);
            ptx::mbar_init(bar_acc_empty(b), Cfg::kEpiWarps * CG);
            ptx::mbar_init(bar_bad_free(b), Cfg::kEpiWarps);
        }
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.tm_p);
        for (int i = 0; i < 3; ++i) ptx::prefetch_tmap(&p.tm_q[i]);
        if (MODE == kTN || MODE == kLoraY) ptx::prefetch_tmap(&p.tm_x);
    }
    if (warp == 1) {
        ptx::tmem_alloc<CG>(ptx::smem_addr(tmem_slot), Cfg::kTmemCols);
        ptx::tmem_relinquish<CG>();
    }
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2) ptx::cluster_sync();
    else __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const bool late = MODE == kNT && !EPI && p.delta != nullptr;
    // With one weight matrix nothing but the operands comes from the kernel before this one: the roles that read or write
    // memory wait for it themselves, and the first weights are asked into L2 meanwhile.
    const bool early = EPI && p.offsets == nullptr;
    if (!late && !early) ptx::griddep_wait();
    if (early) {
        if (threadIdx.x == 0) {
            tab_row[0] = 0;
            tab_row[1] = int32_t(p.rows);
            tab_tile[0] = 0u;
            tab_tile[1] = (p.rows + QCAP - 1u) / QCAP * p.tiles_p;
        }
        __syncthreads();
    } else {
        ragged_table<MODE, QCAP>(p, tab_row, tab_tile);
    }

    const int32_t *list = p.list;
    RaggedWalk<MODE, CG, QCAP, EPI> walk{p,
                                    tab_row,
                                    tab_tile,
                                    list,
                                    blockIdx.x / CG,
                                    gridDim.x / CG,
                                    MODE == kLoraY ? p.tiles_p * p.tiles_q : uniform(tab_tile[p.groups]),
                                    0u,
                                    0u,
                                    0u,
                                    0u,
                                    0u};
    walk.plan_runs();

    // K = 16 steps of K block kb that hold anything (kLoraY: of the projection's)
    auto steps_of = [&](const RaggedSeg &s, uint32_t kb) -> uint32_t {
        const uint32_t left = (MODE == kTN ? s.krows : p.kdim) - kb * kRagBlockK;
        return min(4u, (left + 15u) / 16u);
    };
    // kLoraY: the same of adapter block e, whose columns of b and u start at rank_from(e)
    auto rank_from = [&](uint32_t e) -> uint32_t {
        return p.rank_blocks == 1u ? 0u : (e % p.rank_blocks) * kRagRank;
    };
    auto rank_steps = [&](uint32_t e) -> uint32_t { return min(uint32_t(kRagRank) / 16u, (p.rank - rank_from(e) + 15u) / 16u); };
    // kTN: a last K block that the helper has to finish
    auto fixed_block = [&](const RaggedSeg &s, uint32_t kb) -> bool {
        return MODE == kTN && p.maps == nullptr && kb + 1u == s.kb && (s.krows & 15u) != 0u;
    };

    static_assert(!Cfg::kRegs || Cfg::kRegsFirst + 2 * Cfg::kRegsEpi <= 3 * Cfg::kRegsAll, "registers of the launch");
    if (warp < uint32_t(Cfg::kFirstEpi)) {
    if constexpr (Cfg::kRegs) ptx::regs_dec<Cfg::kRegsFirst>();
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        {
            const bool elected = ptx::elect_one();
            uint32_t stage = 0, phase = 0, fills = 0, tail_uses = 0, last_g = ~0u;
            bool waited = !early;
            walk.template each<true>([&](const RaggedSeg &s) {
                if (EPI && !waited) {
                    const int32_t p0 = int32_t(s.p0 + rank * 128u);
                    if (elected)
                        for (uint32_t v = s.lo; v < min(s.hi, s.lo + uint32_t(STAGES)); ++v) {
                            const int32_t k0 = int32_t(v * kRagBlockK);
                            if constexpr (MODE == kNN) {
                                if (uint32_t(p0) / 64u + 2u <= p.p_groups) ptx::tma_prefetch_4d(&p.tm_p2, 0, k0, p0 / 64, 0);
                            } else {
                                ptx::tma_prefetch_3d(&p.tm_p, k0, p0, 0);
                            }
                        }
                    ptx::griddep_wait();
                    waited = true;
                }
                // kTN: the group's own maps, whose rows end where the group's do
                const CUtensorMap *map_p = &p.tm_p, *map_q = &p.tm_q[0], *map_p2 = &p.tm_p2, *map_q2 = &p.tm_q2;
                if (MODE == kTN && p.maps != nullptr) {
                    map_p = p.maps + 4u * s.g;
                    map_q = map_p + 1;
                    map_p2 = map_p + 2;
                    map_q2 = map_p + 3;
                    if (s.g != last_g && elected) {
                        ptx::tensormap_acquire(map_p);
                        ptx::tensormap_acquire(map_q);
                        if (p.p_groups) ptx::tensormap_acquire(map_p2);
                        if (p.q_groups) ptx::tensormap_acquire(map_q2);
                    }
                    last_g = s.g;
                }
                const uint32_t hq = s.nq / CG;
                // N-side boxes: kTN 64 columns each; otherwise in units of a quarter of the stage's rows, 1, 2, 1 + 2 or 4
                const uint32_t boxes = (hq + 63u) / 64u;
                const uint32_t quarters = (hq + Cfg::kQBox / 4u - 1u) / (Cfg::kQBox / 4u);
                const uint32_t q_bytes = Cfg::kQMn ? boxes * 8192u : quarters * uint32_t(Cfg::kQBox / 4 * 128);
                const int32_t p0 = int32_t(s.p0 + rank * 128u);
                const int32_t q0 = int32_t(s.q0 + rank * hq);
                const bool p_pairs = Cfg::kPMn && uint32_t(p0) / 64u + 2u <= p.p_groups;
                const bool q_pairs = Cfg::kQMn && hq == 128u && uint32_t(q0) / 64u + 2u <= p.q_groups;
                RaggedMix mix(s, p.rank_blocks);
                RaggedNames names(list + size_t(s.g) * p.per, MODE == kLoraY ? s.slots : 0u, MODE == kLoraY ? mix.begun : 0u);
                for (uint32_t v = s.lo; v < s.hi; ++v, ++fills) {
                    const uint32_t e = mix.e, kb = MODE == kLoraY ? mix.m : v;
                    const bool extra = MODE == kLoraY && mix.step();  // adapter block: only P comes by TMA
                    const int32_t adapter = extra ? names[mix.begun - 1u] : 0;
                    if (!ragged_wait_warp<CG>(bar_empty(stage), phase ^ 1u, p, abort_flag, kRagErrEmpty)) return false;
                    const bool tail = extra || fixed_block(s, kb);    // to this CTA's own tail barrier
                    if (elected && !(blockIdx.x == 0 && fills == p.skip_fill && ptx::ld_relaxed_gpu_u32(p.error_word) == 0u)) {
                        const uint32_t p_dst = base + Cfg::kOffP + stage * Cfg::kPBytes;
                        const uint32_t q_dst = base + Cfg::kOffQ + stage * Cfg::kQBytes;
                        const uint32_t bytes = Cfg::kPBytes + (extra ? 0u : q_bytes);
                        rec[4 * stage + 1] = bytes;
                        rec[4 * stage + 2] = bytes * CG;
                        rec[4 * stage + 3] = tail ? 1u | (((tail_uses >> stage) & 1u) << 1) : 0u;
                        rec[4 * stage] = fills + 1u;
                        uint32_t fb = bar_full(stage);
                        if (tail) {
                            if (leader) ptx::mbar_arrive(fb);  // the MMA waits for `fixed` instead
                            fb = bar_tail(stage);
                            ptx::mbar_arrive_expect_tx(fb, bytes);
                        } else {
                            if (leader) ptx::mbar_arrive_expect_tx(fb, bytes * CG);
                            if (CG == 2) fb = ptx::map_to_rank(fb, 0u);
                        }
                        auto load = [&](uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z) {
                            if (CG == 2 && !tail) ptx::tma_load_3d_pair(dst, map, fb, x, y, z);
                            else ptx::tma_load_3d(dst, map, fb, x, y, z);
                        };
                        const int32_t k0 = int32_t(kb * kRagBlockK);
                        auto load2 = [&](uint32_t dst, const CUtensorMap *map, int32_t y, int32_t z, int32_t w) {
                            if (CG == 2 && !tail) ptx::tma_load_4d_pair(dst, map, fb, 0, y, z, w);
                            else ptx::tma_load_4d(dst, map, fb, 0, y, z, w);
                        };
                        if constexpr (MODE == kTN) {
                            const int32_t row = int32_t(s.row0) + k0;
                            if (p_pairs) {
                                load2(p_dst, map_p2, row, p0 / 64, 0);
                            } else {
                                load(p_dst, map_p, p0, row, 0);
                                load(p_dst + 8192u, map_p, p0 + 64, row, 0);
                            }
                            if (q_pairs) {
                                load2(q_dst, map_q2, row, q0 / 64, 0);
                            } else {
                                for (uint32_t b = 0; b < boxes; ++b)
                                    load(q_dst + b * 8192u, map_q, q0 + int32_t(64u * b), row, 0);
                            }
                        } else if (extra) {
                            load(p_dst, &p.tm_x, int32_t(rank_from(e)), p0, adapter);
                        } else {
                            if constexpr (MODE == kNN) {
                                if (p_pairs) {
                                    load2(p_dst, &p.tm_p2, k0, p0 / 64, int32_t(s.g));
                                } else {
                                    load(p_dst, &p.tm_p, p0, k0, int32_t(s.g));
                                    load(p_dst + 8192u, &p.tm_p, p0 + 64, k0, int32_t(s.g));
                                }
                            } else {
                                const int32_t z = MODE == kNT ? int32_t(s.g) : MODE == kLoraU ? int32_t(s.row0) : 0;
                                load(p_dst, &p.tm_p, k0, p0, z);
                            }
                            if (quarters == 4u) {
                                load(q_dst, &p.tm_q[0], k0, q0, 0);
                            } else {
                                if (quarters & 2u) load(q_dst, &p.tm_q[1], k0, q0, 0);
                                if (quarters & 1u) {
                                    const uint32_t from = quarters == 1u ? 0u : uint32_t(Cfg::kQBox) / 2u;
                                    load(q_dst + from * 128u, &p.tm_q[2], k0, q0 + int32_t(from), 0);
                                }
                            }
                        }
                    }
                    if (tail) tail_uses ^= 1u << stage;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                return true;
            });
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (leader) {
            const bool elected = ptx::elect_one();
            const uint32_t tmem_u = uniform(tmem_base);
            const uint32_t idesc0 = ragged_idesc(128u * CG, p.bf16 != 0u, Cfg::kPMn, Cfg::kQMn);
            constexpr uint64_t kPStep = Cfg::kPMn ? (2048u >> 4) : 2u;  // K = 16 inside a swizzle atom, or two 8-row groups
            constexpr uint64_t kQStep = Cfg::kQMn ? (2048u >> 4) : 2u;
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, fixed_uses = 0;
            // K blocks [s.lo, s.hi) into an accumulator
            auto multiply = [&](const RaggedSeg &s) {
                if (!ragged_wait_warp<CG>(bar_acc_empty(acc), acc_phase ^ 1u, p, abort_flag, kRagErrAccEmpty)) return false;
                ptx::tc_fence_after_sync();
                const uint32_t d_tmem = tmem_u + acc * uint32_t(QCAP);
                const uint32_t idesc = idesc0 | ragged_idesc_n(s.nq);
                // K blocks that are full and need no helper come first, four instructions each and nothing else:
                // the issue loop has to stay ahead of the tensor cores
                uint32_t accumulate = 0u;
                const uint32_t whole = (MODE == kTN ? s.krows : p.kdim) / uint32_t(kRagBlockK);
                auto block = [&](uint32_t steps, bool fixed) -> bool {
                    if (!ragged_wait_warp<CG>(bar_full(stage), phase, p, abort_flag, kRagErrFull)) return false;
                    if (Cfg::kHelper && fixed) {
                        if (!ragged_wait_warp<CG>(bar_fixed(stage), (fixed_uses >> stage) & 1u, p, abort_flag, kRagErrFixed))
                            return false;
                        fixed_uses ^= 1u << stage;
                    }
                    ptx::tc_fence_after_sync();
                    const uint64_t p_desc = ragged_desc(base + Cfg::kOffP + stage * Cfg::kPBytes, Cfg::kPMn);
                    const uint64_t q_desc = ragged_desc(base + Cfg::kOffQ + stage * Cfg::kQBytes, Cfg::kQMn);
                    if (elected) {
#pragma unroll
                        for (uint32_t kk = 0; kk < 4u; ++kk)
                            if (kk < steps)
                                ptx::mma_f16<CG>(d_tmem, p_desc + kPStep * kk, q_desc + kQStep * kk, idesc,
                                                 kk == 0u ? accumulate : 1u);
                        if (MODE == kLoraY && fixed) {  // the same of b against u's lower parts
#pragma unroll
                            for (uint32_t kk = 0; kk < uint32_t(kRagRank) / 16u; ++kk)
                                if (kk < steps)
                                    ptx::mma_f16<CG>(d_tmem, p_desc + kPStep * kk, q_desc + kQStep * (kk + kRagRank / 16), idesc, 1u);
                        }
                        if constexpr (CG == 1) ptx::mma_commit(bar_empty(stage));
                        else ptx::mma_commit_pair(bar_empty(stage), uint16_t(3u));
                    }
                    accumulate = 1u;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    return true;
                };
                if (MODE == kLoraY && s.e_hi > s.e_lo) {
                    RaggedMix mix(s, p.rank_blocks);
                    for (uint32_t v = s.lo; v < s.hi; ++v) {
                        const uint32_t e = mix.e, kb = mix.m;
                        const bool extra = mix.step();
                        if (!block(extra ? rank_steps(e) : steps_of(s, kb), extra)) return false;
                    }
                } else {
                    uint32_t kb = MODE == kLoraY ? s.lo - s.e_lo : s.lo;
                    const uint32_t end = MODE == kLoraY ? s.hi - s.e_lo : s.hi;
                    for (; kb < min(end, whole); ++kb)
                        if (!block(4u, false)) return false;
                    for (; kb < end; ++kb)
                        if (!block(steps_of(s, kb), fixed_block(s, kb))) return false;
                }
                if (elected) {
                    if constexpr (CG == 1) ptx::mma_commit(bar_acc_full(acc));
                    else ptx::mma_commit_pair(bar_acc_full(acc), uint16_t(3u));
                }
                if (++acc == 2u) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
                return true;
            };
            walk.template each<true>([&](const RaggedSeg &s) {
                if constexpr (SUM) {
                    RaggedSeg chain = s;
                    for (chain.hi = s.lo; chain.hi < s.hi;) {
                        chain.lo = chain.hi;
                        chain.hi = min(chain.lo + (chain.lo == s.lo ? ragged_first_chain(p, s) : p.chain), s.hi);
                        if (!multiply(chain)) return false;
                    }
                    return true;
                } else {
                    return multiply(s);
                }
            });
            // no MMA may still be running when the tensor memory is freed
            if (elected) {
                if constexpr (CG == 1) ptx::mma_commit(bar_drain);
                else ptx::mma_commit_pair(bar_drain, uint16_t(1u));
                const long long t0 = clock64();
                while (!ptx::mbar_try_wait(bar_drain, 0)) {
                    if (clock64() - t0 > p.wait_limit) {
                        atomicCAS(p.error_word, 0u, kRagErrDrain | (blockIdx.x << 8));
                        break;
                    }
                }
            }
        } else if constexpr (MODE == kLoraY) {
            // ------------------------------------------------ relay
            // What this CTA's helpers have done is made visible in the pair's first CTA, where the MMA issuer waits for it: a
            // release in the cluster takes 1300 to 1800 cycles, which the helpers do not wait for.  One serves two
            // blocks of an adapter.
            uint32_t stage = 0, uses = 0;
            auto advance = [&]() { stage = stage + 1u == STAGES ? 0u : stage + 1u; };
            auto wait_fixed = [&]() {
                const bool ok = ragged_wait_warp<1>(bar_fixed(stage), (uses >> stage) & 1u, p, abort_flag, kRagErrFixed);
                uses ^= 1u << stage;
                return ok;
            };
            walk.template each<true>([&](const RaggedSeg &s) {
                RaggedMix mix(s, p.rank_blocks);
                for (uint32_t v = s.lo; v < s.hi; ++v) {
                    const bool extra = mix.step();
                    const uint32_t at = stage;
                    if (extra && !wait_fixed()) return false;
                    advance();
                    if (!extra) continue;
                    const bool two = mix.run != 0u && v + 1u < s.hi;
                    const uint32_t then = stage;
                    if (two) {
                        mix.step();
                        ++v;
                        if (!wait_fixed()) return false;
                        advance();
                    }
                    if (lane == 0) {
                        ptx::fence_cluster();
                        ptx::mbar_arrive_cluster_relaxed(ptx::map_to_rank(bar_fixed(at), 0u));
                        if (two) ptx::mbar_arrive_cluster_relaxed(ptx::map_to_rank(bar_fixed(then), 0u));
                    }
                    __syncwarp();
                }
                return true;
            });
        }
    }
    } else if (warp < uint32_t(Cfg::kFirstHelper)) {
        // ------------------------------------------------ epilogue
        if constexpr (Cfg::kRegs) ptx::regs_inc<Cfg::kRegsEpi>();
        const uint32_t quarter = warp & 3u;  // tensor-memory lanes [32 quarter, +32)
        const uint32_t set = (warp - uint32_t(Cfg::kFirstEpi)) >> 2;  // its 32-column chunks: set, set + kEpiSets, ...
        const uint32_t buf = base + Cfg::kOffStore + (warp - uint32_t(Cfg::kFirstEpi)) * Cfg::kStoreBytes;
        const bool bf16 = p.bf16 != 0u;
        const uint32_t esize = (MODE == kTN && p.out32) ? 4u : 2u;

        if (early) ptx::griddep_wait();
        // what no tile covers: rows in no group, and the gradients of groups without rows
        {
            const uint64_t first = uint64_t(blockIdx.x) * (32u * Cfg::kEpiWarps) + (threadIdx.x - 32u * Cfg::kFirstEpi);
            const uint64_t stride = uint64_t(gridDim.x) * (32u * Cfg::kEpiWarps);
            auto zero_in = [&](void *out, uint64_t from, uint64_t count) {  // 16-byte chunks
                uint4 *dst = static_cast<uint4 *>(out) + from;
                for (uint64_t i = first; i < count; i += stride) dst[i] = make_uint4(0u, 0u, 0u, 0u);
            };
            auto zero = [&](uint64_t from, uint64_t count) {
                zero_in(p.out, from, count);
                if constexpr (EPI)
                    if (p.kept != nullptr) zero_in(p.kept, from, count);
            };
            if constexpr (MODE == kNT || MODE == kNN) {
                const uint64_t pitch = uint64_t(p.pdim) / 8u;
                const uint32_t head = uint32_t(tab_row[0]), end = uint32_t(tab_row[p.groups]);
                if (head) zero(0, head * pitch);
                if (end < p.rows) zero(end * pitch, (p.rows - end) * pitch);
            }
            if constexpr (MODE == kTN) {
                const uint64_t each = uint64_t(p.pdim) * p.qdim * esize / 16u;
                const uint32_t groups = p.part_rows ? 0u : p.groups;
                for (uint32_t g = 0; g < groups; ++g)
                    if (tab_row[g] == tab_row[g + 1]) zero(g * each, each);
            }
        }

        if (late) ptx::griddep_wait();
        uint32_t acc = 0, acc_phase = 0;
        uint32_t tiles_done = 0;  // SUM
        uint32_t adapted = 0;  // kLoraY: segments with adapter blocks so far
        bool let_in = false;
        bool published = false, taken = false, stopped = false;  // sk: this CTA's flags
        // sk: waits for the partial sums of a tile's earlier K blocks; returns the first worker that has some
        auto wait_partials = [&](const RaggedSeg &s) -> uint32_t {
            const uint32_t w_lo = walk.first_of((s.tile - walk.first_split()) * s.kb);
            if (warp == uint32_t(Cfg::kFirstEpi)) {
                for (uint32_t w = w_lo + lane; w < walk.worker; w += 32u) {
                    uint64_t *flag = p.flags + w * CG + rank;
                    const long long t0 = clock64();
                    uint64_t v;
                    while ((v = ptx::ld_acquire_gpu_u64(flag)) != p.stamp) {
                        if (v == flag_not_coming(p.stamp) || *abort_flag || clock64() - t0 > p.wait_limit) {
                            *abort_flag = 1u;
                            atomicCAS(p.error_word, 0u, kRagErrPartial | (blockIdx.x << 8));
                            break;
                        }
                    }
                    if (v == p.stamp) ptx::st_release_gpu_u64(flag, 0u);
                    else flag_give_up(flag, p.stamp);
                }
                __syncwarp();
            }
            taken = true;
            ptx::named_barrier_sync(1, 32 * Cfg::kEpiWarps);
            return w_lo;
        };
        walk.template each<false>([&](const RaggedSeg &s) {
            const bool split = MODE != kTN && p.sk != 0u && (s.lo != 0u || s.hi != s.kb);
            // what the epilogue takes besides the product is on its way before the product is there
            LinearPiece<EPI> piece_in;
            float bias = 0.0f;
            if constexpr (EPI) {
                const uint32_t prow = s.p0 + rank * 128u + quarter * 32u;
                if (!split || s.hi == s.kb) {
                    if (p.in != nullptr) piece_in.fetch(p.in, p.pdim, s, prow, set);
                    if (MODE == kNT && p.bias != nullptr && prow + lane < p.pdim)
                        bias = ragged_value(static_cast<const uint16_t *>(p.bias)[size_t(s.g) * p.pdim + prow + lane], bf16);
                }
            }
            const uint32_t prow = s.p0 + rank * 128u + quarter * 32u;  // first M-side index of this warp
            const uint32_t chunks = (s.nq + 31u) / 32u;
            // the product's next accumulator is full
            auto arrived = [&]() -> bool {
                const bool ok = ragged_wait<CG>(bar_acc_full(acc), acc_phase, p, abort_flag, kRagErrAccFull);
                // the warps meet at named barriers below when the tile is split or has its columns summed: stop together
                if (MODE != kTN && (SUM || p.sk)) {
                    if (!ptx::named_barrier_and(1, 32 * Cfg::kEpiWarps, ok)) {
                        stopped = true;
                        return false;
                    }
                } else if (!__all_sync(0xffffffffu, ok)) {
                    return false;
                }
                if (!let_in) {
                    ptx::griddep_launch_dependents();
                    let_in = true;
                }
                ptx::tc_fence_after_sync();
                return true;
            };
            if (!arrived()) return false;
            if constexpr (SUM) {
                // the chains are added up in registers, and their sum goes back to tensor memory in the last one's place
                const uint32_t first = ragged_first_chain(p, s);
                if (s.lo + first < s.hi) {
                    constexpr int kOwn = QCAP / 32 / Cfg::kEpiSets;  // 32-column pieces of a warp
                    float run[kOwn][32];
#pragma unroll
                    for (int i = 0; i < kOwn; ++i)
#pragma unroll
                        for (int j = 0; j < 32; ++j) run[i][j] = 0.0f;
                    for (uint32_t next = s.lo + first;; next += p.chain) {
                        const uint32_t column = tmem_base + ((quarter * 32u) << 16) + acc * uint32_t(QCAP);
#pragma unroll
                        for (int i = 0; i < kOwn; ++i) {
                            const uint32_t c = set + uint32_t(i) * Cfg::kEpiSets;
                            if (prow >= p.pdim || c >= chunks) continue;
                            uint32_t r[32];
                            ptx::tmem_ld_32x32b_x32_wait(column + 32u * c, r);
#pragma unroll
                            for (int j = 0; j < 32; ++j) run[i][j] += __uint_as_float(r[j]);
                        }
                        if (next >= s.hi) {
#pragma unroll
                            for (int i = 0; i < kOwn; ++i) {
                                const uint32_t c = set + uint32_t(i) * Cfg::kEpiSets;
                                if (prow < p.pdim && c < chunks) ptx::tmem_st_32x32b_x32(column + 32u * c, run[i]);
                            }
                            ptx::tmem_st_wait();
                            break;
                        }
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (CG == 1) ptx::mbar_arrive(bar_acc_empty(acc));
                            else ptx::mbar_arrive_cluster_signal(ptx::map_to_rank(bar_acc_empty(acc), 0u));
                        }
                        if (++acc == 2u) {
                            acc = 0;
                            acc_phase ^= 1u;
                        }
                        if (!arrived()) return false;
                    }
                }
            }
            const uint32_t t_col = tmem_base + ((quarter * 32u) << 16) + acc * uint32_t(QCAP);
            constexpr uint32_t kSlot = 128u * QCAP;
            // partial tile in the workspace: warp quarter, 32-column chunk, then float4 j of every lane
            const uint32_t piece = quarter * 32u * QCAP + lane * 4u;
            // kLoraY: NaN for the rows whose own adapter holds an infinity or NaN in this lane's row of b
            const bool has_adapters = MODE == kLoraY && s.e_hi > s.e_lo;
            const uint32_t bad_buf = adapted & 1u;
            const bool any = has_adapters && (any_bad[4u * bad_buf] | any_bad[4u * bad_buf + 1u] | any_bad[4u * bad_buf + 2u] |
                                               any_bad[4u * bad_buf + 3u]) != 0u;
            if (has_adapters) ++adapted;
            auto spoil = [&](uint32_t c, uint32_t (&r)[32]) {
                if (!any) return;
                const volatile uint32_t *mask = reinterpret_cast<const volatile uint32_t *>(smem + Cfg::kOffBad + bad_buf * Cfg::kBadBytes);
                for (int32_t i = 0; i < tab_row[s.g]; ++i) {
                    if (!((mask[4 * i + quarter] >> lane) & 1u)) continue;
                    const int32_t adapter = list[size_t(s.g) * p.per + i];
#pragma unroll
                    for (uint32_t j = 0; j < 32u; ++j)
                        if (32u * c + j < s.qn && p.ids[s.q0 + 32u * c + j] == adapter) r[j] = 0x7FC00000u;
                }
            };
            auto release = [&]() {
                if (has_adapters) {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar_bad_free(bad_buf));
                }
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 1) ptx::mbar_arrive(bar_acc_empty(acc));
                    else ptx::mbar_arrive_cluster_signal(ptx::map_to_rank(bar_acc_empty(acc), 0u));
                }
                if (++acc == 2u) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            };
            const bool live = prow < p.pdim;

            // partials move in halves of a chunk, 16 columns: no more than the instruction's N has
            const uint32_t halves = (s.nq + 15u) / 16u;
            if (split && s.hi != s.kb) {
                // ---- publish: the worker with the tile's last K block adds this partial
                if (live) {
                    float *slot = p.partials + size_t(blockIdx.x) * kSlot + piece;
                    for (uint32_t c = set; c < chunks; c += Cfg::kEpiSets) {
                        uint32_t r[32];
                        ptx::tmem_ld_32x32b_x32_wait(t_col + 32u * c, r);
                        if (MODE == kLoraY) spoil(c, r);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (2u * c + uint32_t(j / 4) < halves)
                                ptx::st_global_cg_f4(slot + c * 1024u + j * 128, __uint_as_float(r[4 * j]),
                                                     __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                                                     __uint_as_float(r[4 * j + 3]));
                    }
                }
                release();
                __threadfence();
                ptx::named_barrier_sync(1, 32 * Cfg::kEpiWarps);
                if (threadIdx.x == 32u * Cfg::kFirstEpi) flag_publish(p.flags + blockIdx.x, p.stamp, p.stamp);
                published = true;
                return true;
            }
            uint32_t w_lo = walk.worker;  // workers [w_lo, worker) hold the tile's earlier K blocks
            if (split) w_lo = wait_partials(s);
            // 32 columns of the finished tile: the accumulator plus the other workers' partials, lowest first,
            // two workers' loads in flight
            auto chunk32 = [&](uint32_t c, uint32_t (&r)[32]) {
                ptx::tmem_ld_32x32b_x32_wait(t_col + 32u * c, r);
                if (MODE == kLoraY) spoil(c, r);
                if (MODE != kTN && split) {
                    for (uint32_t w = w_lo; w < walk.worker; w += 2u) {
                        float4 v[2][8];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float *src = p.partials + size_t((w + i) * CG + rank) * kSlot + piece + c * 1024u;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[i][j] = (w + i < walk.worker && 2u * c + uint32_t(j / 4) < halves) ? ptx::ld_global_cg_f4(src + j * 128)
                                                                                                : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                uint32_t *q = r + 4 * j;
                                q[0] = __float_as_uint(__uint_as_float(q[0]) + v[i][j].x);
                                q[1] = __float_as_uint(__uint_as_float(q[1]) + v[i][j].y);
                                q[2] = __float_as_uint(__uint_as_float(q[2]) + v[i][j].z);
                                q[3] = __float_as_uint(__uint_as_float(q[3]) + v[i][j].w);
                            }
                    }
                }
            };
            // low-rank part of this lane's output column, for the rows that have an adapter
            auto load_delta = [&](uint32_t c, float (&d)[32]) {
                const uint32_t t = 32u * c + lane;
                const int32_t id = t < s.qn ? p.ids[s.q0 + t] : -1;
                const uint32_t rows = __ballot_sync(0xffffffffu, uint32_t(id) < p.adapters);
                const float *from = p.delta + size_t(s.q0 + 32u * c) * p.pdim + prow + lane;
                const bool column = prow + lane < p.pdim;
#pragma unroll
                for (uint32_t j = 0; j < 32u; ++j) d[j] = (column && ((rows >> j) & 1u)) ? from[size_t(j) * p.pdim] : 0.0f;
            };
            if constexpr (MODE == kTN) {
                // rows of dw[g] on lanes: boxes of 32 rows x 128 bytes through the swizzled staging buffer
                if (live) {
                    const uint32_t step = p.out32 ? 1u : 2u;  // 32-column chunks per box
                    for (uint32_t c = 0; c < chunks; c += step) {
                        const uint32_t col = s.q0 + 32u * c;
                        uint32_t w[32];
                        if (p.out32) {
                            ptx::tmem_ld_32x32b_x32_wait(t_col + 32u * c, w);
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t r[32];
                                ptx::tmem_ld_32x32b_x32_wait(t_col + 32u * (c + h), r);
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    w[16 * h + j] = ragged_pack(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), bf16);
                            }
                        }
                        if (lane == 0) ptx::bulk_wait_group_read<0>();
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            ptx::st_shared_v4(buf + lane * 128u + ((uint32_t(j) ^ (lane & 7u)) << 4), w[4 * j], w[4 * j + 1],
                                              w[4 * j + 2], w[4 * j + 3]);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            ptx::tma_store_3d(&p.tm_x, buf, int32_t(col), int32_t(prow), int32_t(s.g));
                            ptx::bulk_commit_group();
                        }
                    }
                }
                release();
            } else {
                if (live && MODE == kLoraU) {
                    // a row's values on lanes, a word each: the two parts of u.  Few rows of a tile may have its adapter.
                    const float mul = p.scale ? p.scale[s.row0] : 1.0f;
                    for (uint32_t c = set; c < chunks; c += Cfg::kEpiSets) {
                        const uint32_t t = 32u * c + lane;
                        const uint32_t mine = __ballot_sync(0xffffffffu, (t < s.qn ? p.ids[s.q0 + t] : -1) == int32_t(s.row0));
                        if (mine == 0u) continue;
                        uint32_t r[32];
                        chunk32(c, r);
                        uint32_t *out = static_cast<uint32_t *>(p.out) + size_t(s.q0 + 32u * c) * p.pdim + prow + lane;
                        const uint32_t stored = prow + lane < p.pdim ? mine : 0u;
#pragma unroll
                        for (uint32_t j = 0; j < 32u; ++j) {
                            const float v = __uint_as_float(r[j]) * mul, hi = ragged_unpack(ragged_pack(v, 0.0f, bf16), bf16).x;
                            const uint32_t word = ragged_pack(v, ragged_rest(v, hi), bf16);
                            if ((stored >> j) & 1u) out[j * p.pdim] = word;  // (within a tile: 32 bits)
                        }
                    }
                } else if (EPI && live) {
                    if constexpr (EPI)
                        act::with_kind(p.act, [&](auto kind) {
                            constexpr int kAct = decltype(kind)::value;
                            act::Two both = act::two(0.0f);
                            for (uint32_t c = set; c < chunks; c += Cfg::kEpiSets) {
                                uint32_t r[32], w[16];
                                if (p.in != nullptr) {
                                    piece_in.columns(buf, w);
                                    if (c + Cfg::kEpiSets < chunks) piece_in.fetch(p.in, p.pdim, s, prow, c + Cfg::kEpiSets);
                                } else {
#pragma unroll
                                    for (int i = 0; i < 16; ++i) w[i] = 0u;
                                }
                                chunk32(c, r);
                                if constexpr (MODE == kNT) {
#pragma unroll
                                    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + bias);
                                    if (p.kept != nullptr) linear_store(p.kept, p.pdim, s, prow, c, buf, r, bf16);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        const float2 add = ragged_unpack(w[i], bf16);
                                        const act::Two z = act::two(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                                        const float2 f = act::apart(act::apply<kAct>(z) + act::two(add.x, add.y));
                                        r[2 * i] = __float_as_uint(f.x);
                                        r[2 * i + 1] = __float_as_uint(f.y);
                                    }
                                } else {
#pragma unroll
                                    for (int i = 0; i < 16; ++i) {
                                        const float2 z = ragged_unpack(w[i], bf16);
                                        const act::Two d = act::two(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                                        const float2 f = act::apart(act::apply_grad<kAct>(d, act::two(z.x, z.y)));
                                        r[2 * i] = __float_as_uint(f.x);
                                        r[2 * i + 1] = __float_as_uint(f.y);
                                    }
                                    if constexpr (SUM) {
                                        const uint32_t left = s.qn - 32u * c;  // rows of the tile in this piece and behind it
#pragma unroll
                                        for (uint32_t j = 0; j < 32u; j += 2u)
                                            both = both + act::two(left >= 32u || j < left ? __uint_as_float(r[j]) : 0.0f,
                                                                   left >= 32u || j + 1u < left ? __uint_as_float(r[j + 1]) : 0.0f);
                                    }
                                }
                                linear_store(p.out, p.pdim, s, prow, c, buf, r, bf16);
                            }
                            if constexpr (SUM) {
                                // the two sets of this quarter's warps meet; a sum is read before its place is taken by the next
                                // tile but one
                                const float2 pair = act::apart(both);
                                volatile float *from = reinterpret_cast<volatile float *>(smem + Cfg::kOffSums) + ((tiles_done & 1u) * 128u + quarter * 32u);
                                if (set == 1u) from[lane] = pair.x + pair.y;
                                ptx::named_barrier_sync(2 + quarter, 64);
                                if (set == 0u && prow + lane < p.pdim) {
                                    const uint32_t slot = tab_tile[s.g] / p.tiles_p + s.qi;
                                    p.sums[size_t(slot) * p.pdim + prow + lane] = pair.x + pair.y + from[lane];
                                }
                            }
                        });
                    if constexpr (SUM) ++tiles_done;
                } else if (live) {
                    // rows t on columns: 32 x 32 pieces transposed through shared memory.  A word holds rows
                    // 2i and 2i + 1 of one output column; a lane reads four columns' words and takes them apart.
                    char *out = static_cast<char *>(p.out);
                    const uint32_t col = prow + 4u * (lane & 7u);
                    for (uint32_t c = set; c < chunks; c += Cfg::kEpiSets) {
                        uint32_t r[32];
                        float d[MODE == kNT ? 32 : 1];
                        if constexpr (MODE == kNT)
                            if (late) load_delta(c, d);  // on its way while the partials come
                        chunk32(c, r);
                        if constexpr (MODE == kNT)
                            if (late) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + d[j]);
                            }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            ptx::st_shared_u32(buf + uint32_t(i) * 128u + lane * 4u,
                                               ragged_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), bf16));
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t pr = uint32_t(i) * 4u + (lane >> 3);
                            const uint4 v = ptx::ld_shared_v4(buf + pr * 128u + (lane & 7u) * 16u);
                            const uint32_t row = 32u * c + 2u * pr;  // in the tile
                            if (col < p.pdim) {
#pragma unroll
                                for (uint32_t h = 0; h < 2u; ++h) {
                                    if (row + h >= s.qn) continue;
                                    const uint32_t sel = h ? 0x7632u : 0x5410u;
                                    ptx::st_global_v2(out + (size_t(s.q0 + row + h) * p.pdim + col) * 2u,
                                                      __byte_perm(v.x, v.y, sel), __byte_perm(v.z, v.w, sel));
                                }
                            }
                        }
                    }
                }
                release();
            }
            return true;
        });
        if (MODE == kTN && lane == 0) ptx::bulk_wait_group<0>();
        if (MODE != kTN && stopped && p.sk && warp == uint32_t(Cfg::kFirstEpi)) walk.leave_flags(rank, published, taken);
        if constexpr (Cfg::kRegs) ptx::regs_dec<Cfg::kRegsFirst>();  // (as the others: one teardown for all)
    } else if constexpr (Cfg::kHelper) {
        // ------------------------------------------------ helper
        // Four warps that share a stage's rows and never wait for each other: `fixed` counts them all.
        const uint32_t tid = threadIdx.x - 32u * uint32_t(Cfg::kFirstHelper);
        const uint32_t part = tid >> 5;
        uint32_t fills = 0, tail_uses = 0, adapted = 0;
        auto wait_tail = [&](uint32_t stage) {
            const bool ok = ragged_wait_warp<1>(bar_tail(stage), (tail_uses >> stage) & 1u, p, abort_flag, kRagErrTail);
            tail_uses ^= 1u << stage;
            return ok;
        };
        auto hand_over = [&](uint32_t stage) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 1 || MODE == kLoraY) ptx::mbar_arrive(bar_fixed(stage));
                else ptx::mbar_arrive_cluster(ptx::map_to_rank(bar_fixed(stage), 0u));
            }
        };
        walk.template each<false>([&](const RaggedSeg &s) {
            const uint32_t hq = s.nq / CG;
            const uint32_t first = fills;
            fills += s.hi - s.lo;
            if constexpr (MODE == kTN) {
                if (!fixed_block(s, s.kb - 1u)) return true;
                const uint32_t stage = (fills - 1u) % STAGES;
                if (!wait_tail(stage)) return false;
                const uint32_t from = s.krows % kRagBlockK, to = (from + 15u) & ~15u;
                const uint32_t boxes = (hq + 63u) / 64u;
                const uint32_t lines = (to - from) * 8u;  // 16-byte pieces of the rows to clear, per 64-column box
                for (uint32_t i = tid; i < lines * (2u + boxes); i += kRagHelpers) {
                    const uint32_t b = i / lines;
                    const uint32_t at = (b < 2u ? base + Cfg::kOffP + stage * Cfg::kPBytes + b * 8192u
                                                : base + Cfg::kOffQ + stage * Cfg::kQBytes + (b - 2u) * 8192u) +
                                        from * 128u + (i - b * lines) * 16u;
                    ptx::st_shared_v4(at, 0u, 0u, 0u, 0u);
                }
                hand_over(stage);
            } else {
                // adapter blocks: rows of this CTA's part of the tile, u where the row has the slot's adapter
                if (s.e_hi <= s.e_lo) return true;
                static_assert(Cfg::kQCta <= kRagHelpers, "one row of u per helper thread");
                const uint32_t row = s.q0 + rank * hq + tid;
                const int32_t id = (tid < hq && rank * hq + tid < s.qn) ? p.ids[row] : -1;
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.u) + size_t(row) * p.rank * 4u);
                constexpr uint32_t kHalf = kRagRank / 8;  // 16-byte pieces of either part of u in a block
                RaggedNames names(list + size_t(s.g) * p.per, s.slots, s.e_lo / p.rank_blocks);
                uint4 u0[2 * kHalf], u1[2 * kHalf];  // of the first two blocks (rank <= 64: of all), or of the present ones
                auto fetch = [&](uint32_t column, uint4 (&u)[2 * kHalf]) {
#pragma unroll
                    for (uint32_t c = 0; c < kHalf; ++c) {
                        const uint32_t at = column + 8u * c;
                        const bool there = uint32_t(id) < p.adapters && at < p.rank;
                        const uint4 v = there ? src[at / 4u] : make_uint4(0u, 0u, 0u, 0u);
                        const uint4 w = there ? src[at / 4u + 1u] : make_uint4(0u, 0u, 0u, 0u);
                        u[c] = make_uint4(__byte_perm(v.x, v.y, 0x5410u), __byte_perm(v.z, v.w, 0x5410u),
                                          __byte_perm(w.x, w.y, 0x5410u), __byte_perm(w.z, w.w, 0x5410u));
                        u[c + kHalf] = make_uint4(__byte_perm(v.x, v.y, 0x7632u), __byte_perm(v.z, v.w, 0x7632u),
                                                  __byte_perm(w.x, w.y, 0x7632u), __byte_perm(w.z, w.w, 0x7632u));
                    }
                };
                fetch(0u, u0);
                fetch(kRagRank, u1);
                // the table of b rows with infinities is free once the epilogue is done with the tile before last;
                // each warp keeps the words of its own rows
                const uint32_t bad_buf = adapted & 1u;
                if (!ragged_wait_warp<1>(bar_bad_free(bad_buf), ((adapted >> 1) & 1u) ^ 1u, p, abort_flag, kRagErrFixed))
                    return false;
                ++adapted;
                uint32_t *mask = reinterpret_cast<uint32_t *>(smem + Cfg::kOffBad + bad_buf * Cfg::kBadBytes);
                for (uint32_t i = lane; i < uint32_t(tab_row[s.g]); i += 32u) mask[4u * i + part] = 0u;
                if (lane == 0) any_bad[4u * bad_buf + part] = 0u;
                __syncwarp();
                // exponent bits of both halves of a word; all ones (infinity or NaN) carry into the top bit
                const uint32_t expo = p.bf16 ? 0x7F807F80u : 0x7C007C00u;
                const uint32_t carry = p.bf16 ? 0x00800080u : 0x04000400u;
                // adapter number `slot` is item ceil((slot + 1) items / slots) - 1
                const uint32_t items = s.kb - s.extra + s.slots;
                uint32_t slot = p.rank_blocks == 1u ? s.e_lo : s.e_lo / p.rank_blocks;
                const uint64_t scaled = uint64_t(slot + 1u) * items;
                uint32_t quot = uint32_t(scaled / s.slots), rest = uint32_t(scaled - uint64_t(quot) * s.slots);
                const uint32_t quot_step = items / s.slots, rest_step = items - quot_step * s.slots;
                for (uint32_t e = s.e_lo; e < s.e_hi;) {
                    const uint32_t stage = (first + quot + (rest ? 1u : 0u) - 1u + e - slot - s.lo) % STAGES;
                    const bool mine = id == names[slot];
                    const uint32_t sub = e - slot * p.rank_blocks;
                    const bool second = sub == 1u && p.rank_blocks == 2u;
                    if (mine && p.rank_blocks > 2u) fetch(sub * kRagRank, u0);
                    // b has landed, so the stage is free: the producer waited for that.  (The stage's empty barrier
                    // cannot be waited for here: it may be more than one phase away.)
                    if (!wait_tail(stage)) return false;
                    // u where the row has the slot's adapter, zeros elsewhere
                    const uint32_t q_at = base + Cfg::kOffQ + stage * Cfg::kQBytes + tid * 128u;
                    if (tid < hq) {
#pragma unroll
                        for (uint32_t c = 0; c < 2u * kHalf; ++c) {
                            uint4 v = second ? u1[c] : u0[c];
                            if (!mine) v = make_uint4(0u, 0u, 0u, 0u);
                            ptx::st_shared_v4(q_at + ((c ^ (tid & 7u)) << 4), v.x, v.y, v.z, v.w);
                        }
                    }
                    // b's row tid: zeros for infinities and NaN, which the other adapters' zero rows of u would turn into NaN
                    const uint32_t p_at = base + Cfg::kOffP + stage * Cfg::kPBytes + tid * 128u;
                    uint32_t odd = 0u;
#pragma unroll
                    for (uint32_t c = 0; c < kHalf; ++c) {
                        const uint4 v = ptx::ld_shared_v4(p_at + ((c ^ (tid & 7u)) << 4));
                        odd |= ((v.x & expo) + carry) | ((v.y & expo) + carry) | ((v.z & expo) + carry) | ((v.w & expo) + carry);
                    }
                    if (odd & 0x80008000u) {
#pragma unroll 1
                        for (uint32_t c = 0; c < kHalf; ++c) {
                            const uint32_t at = p_at + ((c ^ (tid & 7u)) << 4);
                            const uint4 v = ptx::ld_shared_v4(at);
                            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t top = ((w[j] & expo) + carry) & 0x80008000u;
                                w[j] &= ((top & 0x8000u) ? 0xFFFF0000u : 0xFFFFFFFFu) & ((top & 0x80000000u) ? 0x0000FFFFu : 0xFFFFFFFFu);
                            }
                            ptx::st_shared_v4(at, w[0], w[1], w[2], w[3]);
                        }
                        atomicOr(mask + 4u * slot + part, 1u << lane);
                        any_bad[4u * bad_buf + part] = 1u;
                    }
                    hand_over(stage);
                    ++e;
                    if (e == (slot + 1u) * p.rank_blocks) {
                        ++slot;
                        quot += quot_step;
                        rest += rest_step;
                        if (rest >= s.slots) {
                            rest -= s.slots;
                            ++quot;
                        }
                    }
                }
            }
            return true;
        });
    }

    // ---------------------------------------------------- teardown
    ptx::griddep_launch_dependents();
    // (a kernel that ends counts as the end of those before it)
    if (late || early) ptx::griddep_wait();
    __syncwarp();
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2) ptx::cluster_sync();
    else __syncthreads();
    ptx::tc_fence_after_sync();
    if (threadIdx.x == 0) {
        bool aborted = *abort_flag != 0u;
        if constexpr (CG == 2)
            aborted = ptx::ld_shared_cluster_u32(ptx::map_to_rank(base + Cfg::kOffAbort, 0u)) != 0u ||
                      ptx::ld_shared_cluster_u32(ptx::map_to_rank(base + Cfg::kOffAbort, 1u)) != 0u;
        if (aborted) ragged_drain<STAGES, CG>(base + Cfg::kOffBar, base + Cfg::kOffRec, leader, p);
    }
    if constexpr (CG == 2) ptx::cluster_sync();
    if (warp == 1) ptx::tmem_dealloc<CG>(tmem_base, Cfg::kTmemCols);
}

}  // namespace gemm_f16
