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
    uint32_t sk;             // 1: equal runs of K-block iterations
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

template <int MODE, int CG, int QCAP, int STAGES>
struct RaggedCfg {
    static_assert(CG == 1 || CG == 2, "cta group");
    static constexpr bool kPMn = (MODE == kNN || MODE == kTN);  // M-side operand MN-major
    static constexpr bool kQMn = (MODE == kTN);                 // N-side operand MN-major
    static constexpr bool kHelper = (MODE == kTN || MODE == kLoraY);
    // (kTN: eight warps' boxes of 128 bytes a row do not fit; of 64 bytes, or shared by two warps, they took 8 and
    // 2% longer than four for 16384 rows, 32 groups, 4096 x 4096)
    static constexpr int kEpiSets = (QCAP == 256 && MODE != kTN) ? 2 : 1;
    static constexpr int kEpiWarps = 4 * kEpiSets;
    static constexpr int kFirstHelper = 2 + kEpiWarps;          // warp
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
    static constexpr int kSmemBytes = kOffAnyBad + 32 + 1024;
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

template <int MODE, int CG, int QCAP>
struct RaggedWalk {
    const RaggedParams &p;
    const int32_t *tab_row;    // offsets (groups + 1), or counts per row tile
    const uint32_t *tab_tile;  // tiles before each group (groups + 1)
    const int32_t *list;       // kLoraU, kLoraY: the adapters of each row tile
    uint32_t worker, workers, total;
    uint32_t run, longer;      // sk: K-block iterations of a worker; the first `longer` workers have one more
    uint32_t tile_blocks;      // sk: K blocks of every tile

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
        const uint32_t iters = total * tile_blocks;  // below 2^32: the host checks
        const uint32_t most = max(1u, iters / kMinRun);
        if (most < workers) workers = most;
        run = iters / workers;
        longer = iters - run * workers;
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
        if (total == 0u || worker >= workers) return;
        const uint32_t begin = run_begin(worker);
        uint32_t it = run_begin(worker + 1u);
        const uint32_t kb = tile_blocks;
        while (it > begin) {
            const uint32_t u = (it - 1u) / kb;
            const uint32_t start = u * kb;
            decode(u, s, near);
            s.lo = begin > start ? begin - start : 0u;
            s.hi = it - start;
            const uint32_t lo = s.lo;
            count_extra(s);
            if constexpr (UNIFORM) uniform<MODE>(s);
            if (!f(s)) return;
            it = start + lo;
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

template <int MODE, int CG, int QCAP, int STAGES>
__global__ void __launch_bounds__(RaggedCfg<MODE, CG, QCAP, STAGES>::kThreads, 1) gemm_ragged_kernel(const __grid_constant__ RaggedParams p)
{
    using Cfg = RaggedCfg<MODE, CG, QCAP, STAGES>;
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
    const bool late = MODE == kNT && p.delta != nullptr;
    if (!late) ptx::griddep_wait();
    ragged_table<MODE, QCAP>(p, tab_row, tab_tile);

    const int32_t *list = p.list;
    RaggedWalk<MODE, CG, QCAP> walk{p,
                                    tab_row,
                                    tab_tile,
                                    list,
                                    blockIdx.x / CG,
                                    gridDim.x / CG,
                                    MODE == kLoraY ? p.tiles_p * p.tiles_q : uniform(tab_tile[p.groups]),
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

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        {
            const bool elected = ptx::elect_one();
            uint32_t stage = 0, phase = 0, fills = 0, tail_uses = 0, last_g = ~0u;
            walk.template each<true>([&](const RaggedSeg &s) {
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
            walk.template each<true>([&](const RaggedSeg &s) {
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
    } else if (warp < uint32_t(Cfg::kFirstHelper)) {
        // ------------------------------------------------ epilogue
        const uint32_t quarter = warp & 3u;  // tensor-memory lanes [32 quarter, +32)
        const uint32_t set = (warp - 2u) >> 2;  // its 32-column chunks: set, set + kEpiSets, ...
        const uint32_t buf = base + Cfg::kOffStore + (warp - 2u) * Cfg::kStoreBytes;
        const bool bf16 = p.bf16 != 0u;
        const uint32_t esize = (MODE == kTN && p.out32) ? 4u : 2u;

        // what no tile covers: rows in no group, and the gradients of groups without rows
        {
            const uint64_t first = uint64_t(blockIdx.x) * (32u * Cfg::kEpiWarps) + (threadIdx.x - 64u);
            const uint64_t stride = uint64_t(gridDim.x) * (32u * Cfg::kEpiWarps);
            auto zero = [&](uint64_t from, uint64_t count) {  // 16-byte chunks
                uint4 *dst = static_cast<uint4 *>(p.out) + from;
                for (uint64_t i = first; i < count; i += stride) dst[i] = make_uint4(0u, 0u, 0u, 0u);
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
        uint32_t adapted = 0;  // kLoraY: segments with adapter blocks so far
        bool let_in = false;
        bool published = false, taken = false, stopped = false;  // sk: this CTA's flags
        walk.template each<false>([&](const RaggedSeg &s) {
            const bool ok = ragged_wait<CG>(bar_acc_full(acc), acc_phase, p, abort_flag, kRagErrAccFull);
            const bool split = MODE != kTN && p.sk != 0u && (s.lo != 0u || s.hi != s.kb);
            // the warps meet at named barriers below when the tile is split: stop together
            if (MODE != kTN && p.sk) {
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
            const uint32_t t_col = tmem_base + ((quarter * 32u) << 16) + acc * uint32_t(QCAP);
            const uint32_t prow = s.p0 + rank * 128u + quarter * 32u;  // first M-side index of this warp
            const uint32_t chunks = (s.nq + 31u) / 32u;
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
                if (threadIdx.x == 64u) flag_publish(p.flags + blockIdx.x, p.stamp, p.stamp);
                published = true;
                return true;
            }
            uint32_t w_lo = walk.worker;  // workers [w_lo, worker) hold the tile's earlier K blocks
            if (split) {
                w_lo = walk.first_of(s.tile * s.kb);
                if (warp == 2u) {
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
            }
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
        if (MODE != kTN && stopped && warp == 2u) walk.leave_flags(rank, published, taken);
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
    if (late) ptx::griddep_wait();
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

// kTN: every group's tensor maps with the rows ending at the group's end, so that TMA fills the rest of its last K block
// with zeros (32 uneven groups of 16384 rows in all, 4096 x 4096: 442 us with the helper zeroing each tile's last
// block, 358 so).  One block per group, one warp per map; some 3 us in front of the product.
struct RaggedMapsParams {
    CUtensorMap maps[4];
    const int32_t *offsets;
    uint32_t groups, rows;
    uint32_t have;      // bit i: maps[i] is one
    CUtensorMap *out;   // [groups][4]
};

__global__ void __launch_bounds__(128) ragged_maps_kernel(const __grid_constant__ RaggedMapsParams p)
{
    __shared__ __align__(128) CUtensorMap s_map[4];
    ptx::griddep_wait();
    const uint32_t lane = threadIdx.x & 31u, i = threadIdx.x >> 5, g = blockIdx.x;
    // the group's end as ragged_table has it: the largest of the clamped offsets up to it
    int32_t end = 0;
    for (uint32_t k = lane; k <= g + 1u; k += 32u) end = max(end, min(p.offsets[k], int32_t(p.rows)));
    end = __reduce_max_sync(0xffffffffu, end);
    if ((p.have >> i) & 1u) {
        reinterpret_cast<uint32_t *>(&s_map[i])[lane] = reinterpret_cast<const uint32_t *>(&p.maps[i])[lane];
        __syncwarp();
        if (lane == 0) ptx::tensormap_set_dim1(ptx::smem_addr(&s_map[i]), uint32_t(max(end, 1)));
        __syncwarp();
        ptx::tensormap_publish(p.out + 4u * g + i, ptx::smem_addr(&s_map[i]));
    }
    ptx::griddep_launch_dependents();
}

// kTN with few tiles: the rows of a group are cut into parts of `part_rows` (a multiple of a K block), each part's sum
// goes to a matrix of its own in fp32, and this kernel adds a group's parts, in order, and rounds once.  Bound by L2 for
// large matrices, else by its launch.  One block row per group.  (10560 rows in one group, 64 x 248: 63.6 us whole, 15.6
// in parts; 27407 rows in 3 groups, 640 x 104: 89.3 and 18.7; 9426 in 2, 144 x 3328: 32.6 and 25.3.)
constexpr uint32_t kRagPartGroups = 128;

struct RaggedPartsParams {
    const float4 *parts;  // [parts][n * k / 4]
    const int32_t *offsets;
    void *out;            // [groups, n, k]
    uint32_t groups, rows, part_rows;
    uint32_t quads;       // n * k / 4
    uint32_t out32, bf16;
};

__global__ void __launch_bounds__(256) ragged_parts_kernel(const __grid_constant__ RaggedPartsParams p)
{
    __shared__ int32_t s_row[kRagPartGroups + 1];
    __shared__ uint32_t s_parts[kRagPartGroups];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t i = threadIdx.x, g = blockIdx.y;
    if (i <= p.groups) s_row[i] = max(0, min(p.offsets[i], int32_t(p.rows)));
    __syncthreads();
    if (i < p.groups) {  // as ragged_table has them
        int32_t begin = 0;
        for (uint32_t j = 0; j <= i; ++j) begin = max(begin, s_row[j]);
        s_parts[i] = uint32_t((max(begin, s_row[i + 1]) - begin + int32_t(p.part_rows) - 1) / int32_t(p.part_rows));
    }
    __syncthreads();
    uint32_t first = 0;
    for (uint32_t j = 0; j < g; ++j) first += s_parts[j];
    const uint32_t count = s_parts[g];
    const uint32_t q = blockIdx.x * 256u + i;
    if (q >= p.quads) return;
    const float4 *from = p.parts + size_t(first) * p.quads + q;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (uint32_t j = 0; j < count; ++j) {
        const float4 v = from[size_t(j) * p.quads];
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    const size_t at = size_t(g) * p.quads + q;
    if (p.out32)
        static_cast<float4 *>(p.out)[at] = sum;
    else
        static_cast<uint2 *>(p.out)[at] = make_uint2(ragged_pack(sum.x, sum.y, p.bf16 != 0u), ragged_pack(sum.z, sum.w, p.bf16 != 0u));
}

// Adapters without the tensor cores: with an adapter to nearly every row, all of the work is reading a and b once, and
// each row sees its own adapter only.  u = scale x a^T and delta = u b^T stay in fp32.  They run beside the projection,
// which starts at once and waits for delta in its epilogue.  16 rows with 16 adapters of rank 16, 8192 x 4096, take 22 us,
// as without adapters 20; 64 with 64 take 30 (as K blocks of the projection 36): there the two kernels, 7 us each on an
// idle GPU, end after the projection's loads.
//
// For a few rows of a low rank a cluster of eight CTAs takes a row through both steps and trades u through distributed
// shared memory: one launch fewer, 2 to 4 us of the host's time, and the GPU's with it, then by the two kernels: 16 rows,
// rank 16, 8192 x 4096, 21.7 us and 23.6; 32 rows 23.1 and 24.7; 1 row, 4096 x 4096, 14.4 and 13.9.  But 64 rows take 32.6
// and 29.0, and rank 64 (16 rows, 11008 x 4096) 35.8 and 33.3: a row's work on eight SMs only.
struct LoraFewParams {
    const void *x, *a, *b;
    const int32_t *ids;
    const float *scale;
    float *u;       // [rows, rank]
    float *delta;   // [rows, n]
    uint32_t rows, n, k, rank, adapters, bf16;
};

// Four of a row's u's (before the scale) by WARPS warps that share k: each lane multiplies 8 elements at a time.  The sums
// of a single warp are in all lanes; of four, thread t returns number t mod 4, and s_sum is the block's.
template <int WARPS>
__device__ __forceinline__ float lora_dot4(const LoraFewParams &p, uint32_t row, int32_t id, uint32_t r0, float (*s_sum)[4])
{
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const bool bf16 = p.bf16 != 0u;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.x) + size_t(row) * p.k * 2u);
    const char *a = static_cast<const char *>(p.a) + (size_t(id) * p.rank + r0) * p.k * 2u;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (uint32_t i = WARPS == 1 ? lane : threadIdx.x; i < p.k / 8u; i += 32u * WARPS) {
        const uint4 xv = x[i];
        uint4 av[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) av[r] = reinterpret_cast<const uint4 *>(a + size_t(r) * p.k * 2u)[i];
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 xf = ragged_unpack(xw[j], bf16);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t aw = j == 0 ? av[r].x : j == 1 ? av[r].y : j == 2 ? av[r].z : av[r].w;
                const float2 af = ragged_unpack(aw, bf16);
                sum[r] = fmaf(xf.x, af.x, sum[r]);
                sum[r] = fmaf(xf.y, af.y, sum[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], d);
    const uint32_t r = threadIdx.x & 3u;
    if constexpr (WARPS == 1) {
        return r == 0u ? sum[0] : r == 1u ? sum[1] : r == 2u ? sum[2] : sum[3];
    } else {
        __syncthreads();  // the four before have been read
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) s_sum[warp][i] = sum[i];
        __syncthreads();
        return (s_sum[0][r] + s_sum[1][r]) + (s_sum[2][r] + s_sum[3][r]);
    }
}

// 128 columns of a row's delta by one warp.  LANES lanes share a row of b, 16 bytes each, with their part of u in
// registers; eight rows' loads are in flight.  (One lane to a row of b read a line per lane and load.)
template <int LANES>
__device__ __forceinline__ void lora_columns(const LoraFewParams &p, uint32_t row, int32_t id, uint32_t col0, const float (&u)[8])
{
    const uint32_t lane = threadIdx.x & 31u, part = lane % LANES;
    const bool bf16 = p.bf16 != 0u, live = 8u * part < p.rank;
    constexpr uint32_t kRows = 32 / LANES;  // rows of b a warp reads at a time
    constexpr uint32_t kFlight = 8;         // and such reads in flight
    const char *b = static_cast<const char *>(p.b) + size_t(id) * p.n * p.rank * 2u + 16u * part;
#pragma unroll 1
    for (uint32_t i0 = 0; i0 < 128u; i0 += kFlight * kRows) {
        uint4 v[kFlight];
#pragma unroll
        for (int i = 0; i < int(kFlight); ++i) {
            const uint32_t col = col0 + i0 + uint32_t(i) * kRows + lane / LANES;
            v[i] = (live && col < p.n && i0 + uint32_t(i) * kRows < 128u)
                       ? *reinterpret_cast<const uint4 *>(b + size_t(col) * p.rank * 2u)
                       : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < int(kFlight); ++i) {
            if (i0 + uint32_t(i) * kRows >= 128u) continue;
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = ragged_unpack(w[j], bf16);
                sum = fmaf(f.x, u[2 * j], sum);
                sum = fmaf(f.y, u[2 * j + 1], sum);
            }
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const uint32_t col = col0 + i0 + uint32_t(i) * kRows + lane / LANES;
            if (part == 0u && col < p.n) p.delta[size_t(row) * p.n + col] = sum;
        }
    }
}

// An item is a row and four of its u's: a block's (WARPS = 4), or, where there are more of them than the GPU has blocks at
// a time, a warp's.  (Here and below items are counted in 32 bits: rows that have more go by the tensor cores.)
template <int WARPS>
__global__ void __launch_bounds__(128) lora_shrink_kernel(const __grid_constant__ LoraFewParams p)
{
    __shared__ float s_sum[4][4];
    ptx::griddep_wait();
    // (after the wait: what the next kernels read from before this one is complete as well)
    ptx::griddep_launch_dependents();
    constexpr uint32_t kItems = 4 / WARPS;  // of a block at a time
    const uint32_t parts = p.rank / 4u;
    for (uint32_t item = blockIdx.x * kItems + (WARPS == 1 ? threadIdx.x >> 5 : 0u); item < p.rows * parts; item += gridDim.x * kItems) {
        const uint32_t row = item / parts, r0 = (item - row * parts) * 4u;
        const int32_t id = p.ids[row];
        if (uint32_t(id) >= p.adapters) continue;
        const float v = lora_dot4<WARPS>(p, row, id, r0, s_sum) * (p.scale ? p.scale[id] : 1.0f);
        const uint32_t t = WARPS == 1 ? threadIdx.x & 31u : threadIdx.x;
        if (t < 4u) p.u[size_t(row) * p.rank + r0 + t] = v;
    }
}

// An item, a warp's, is a row and 128 of its columns.
template <int LANES>
__global__ void __launch_bounds__(128) lora_expand_kernel(const __grid_constant__ LoraFewParams p)
{
    // The product behind this kernel reads nothing of the kernel before this one; that one has waited for all before it.
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const uint32_t part = (threadIdx.x & 31u) % LANES, parts = (p.n + 127u) / 128u;
    for (uint32_t item = blockIdx.x * 4u + (threadIdx.x >> 5); item < p.rows * parts; item += gridDim.x * 4u) {
        const uint32_t row = item / parts;
        const int32_t id = p.ids[row];
        if (uint32_t(id) >= p.adapters) continue;
        float u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 8u * part < p.rank ? p.u[size_t(row) * p.rank + 8u * part + j] : 0.0f;
        lora_columns<LANES>(p, row, id, (item - row * parts) * 128u, u);
    }
}

// Both steps of one row by a cluster.
constexpr uint32_t kLoraCluster = 8;

template <int LANES>
__global__ void __launch_bounds__(128) lora_rows_kernel(const __grid_constant__ LoraFewParams p)
{
    __shared__ float s_sum[4][4];
    __shared__ float s_u[32];
    ptx::cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();  // (after the wait, as above)
    const uint32_t part = (threadIdx.x & 31u) % LANES, rank = ptx::cluster_ctarank(), row = blockIdx.x / kLoraCluster;
    const int32_t id = p.ids[row];
    if (uint32_t(id) >= p.adapters) return;  // (the same for the whole cluster)
    for (uint32_t r0 = 4u * rank; r0 < p.rank; r0 += 4u * kLoraCluster) {
        const float v = lora_dot4<4>(p, row, id, r0, s_sum) * (p.scale ? p.scale[id] : 1.0f);
        if (threadIdx.x < 4u * kLoraCluster)  // four values to every CTA
            ptx::st_shared_cluster_u32(ptx::map_to_rank(ptx::smem_addr(&s_u[r0 + (threadIdx.x & 3u)]), threadIdx.x >> 2),
                                       __float_as_uint(v));
    }
    __syncwarp();
    ptx::cluster_sync();
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = 8u * part < p.rank ? s_u[8u * part + j] : 0.0f;
    for (uint32_t item = rank * 4u + (threadIdx.x >> 5); item < (p.n + 127u) / 128u; item += 4u * kLoraCluster)
        lora_columns<LANES>(p, row, id, item * 128u, u);
}

// Lists for the tensor cores' form: the adapters present in each tile of `per` rows (per <= 256), in order of first
// appearance.  Rows with an id outside [0, adapters) have none.  Two cuttings of the same rows at once: `tiles` blocks for
// the first, the rest for the second.  Bound by latency, some 4 us.
struct LoraListParams {
    const int32_t *ids;
    uint32_t rows, adapters, tiles;
    uint32_t per[2];
    int32_t *counts[2], *list[2];
};

__global__ void __launch_bounds__(256) lora_list_kernel(const __grid_constant__ LoraListParams p)
{
    __shared__ __align__(16) int32_t s_id[256];
    __shared__ uint32_t s_warp[8];
    ptx::griddep_wait();
    const uint32_t cut = blockIdx.x < p.tiles ? 0u : 1u, tile = blockIdx.x - cut * p.tiles, per = p.per[cut];
    const uint32_t t = threadIdx.x, row = tile * per + t;
    int32_t id = (p.adapters != 0u && t < per && row < p.rows) ? p.ids[row] : -1;
    if (uint32_t(id) >= p.adapters) id = -1;
    s_id[t] = id;
    __syncthreads();
    // the first row with its id: every earlier one differs (four at a time, the same words for the whole warp)
    bool first = id >= 0;
    for (uint32_t i = 0; i < (t | 31u) + 1u; i += 4u) {
        const int4 v = *reinterpret_cast<const int4 *>(s_id + i);
        first &= !((v.x == id && i < t) || (v.y == id && i + 1u < t) || (v.z == id && i + 2u < t) || (v.w == id && i + 3u < t));
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, first);
    if ((t & 31u) == 0) s_warp[t >> 5] = __popc(vote);
    __syncthreads();
    uint32_t at = __popc(vote & ((1u << (t & 31u)) - 1u)), total = 0;
    for (uint32_t w = 0; w < 8u; ++w) {
        if (w < (t >> 5)) at += s_warp[w];
        total += s_warp[w];
    }
    if (first) p.list[cut][size_t(tile) * per + at] = id;
    if (t == 0) p.counts[cut][tile] = int32_t(total);
    ptx::griddep_launch_dependents();
}

}  // namespace gemm_f16
