// pkv_mass.cu -- attention weight that every cached token receives, added up
// over a step's queries and a kv head's query heads, on the 5th-generation
// tensor cores (tcgen05, TMEM accumulators).
//
// What it computes.  mass[t] += sum over the (query, head) columns c that see
// slot t of exp2((k_t . q_c scale - lse_c) log2(e)).  The lse is given, so
// there is no running maximum and nothing to rescale: S^T = K Q^T with the keys
// on the MMA's rows, so that a TMEM lane is a key and a thread adds up its own
// key's columns in a register.  No value crosses threads, and what a NaN in one
// key or one column does stays there.
//
// What bounds it.  A decode step reads K once (32 KB for 128 keys at head_dim
// 128, 0.74 us of an SM's share of the measured HBM rate) for 8 MMAs of 128 x 16
// x 16: memory.  64 uneven rows of 95,000 tokens in all, one of 32,768, take 39
// us, 5.1 TB/s; while it streams it runs at 93 % of the copy rate, and the first
// MMA comes 6.6 us after a CTA has begun (5.0 until its range and pages are known
// and the first copy leaves, 1.6 until its data is there).  One token over 64: 7.5 us.
// With many queries 128 keys x 128 columns (a pair) are 8 MMAs of 128 x 128 x 16,
// 512 cycles at the tensor pipe's nominal rate, and 16,384 exponentials, 512
// cycles at the 32 a cycle measured; a pair takes about 990.  No unit is full
// (tensor 43 %, exponentials 43 %, issue slots 57 % of the elapsed cycles): a pair
// goes from the MMAs to the sums and back in 3,990 cycles, and TMEM holds four.
// Of those the sums take 2,580 (four TMEM loads at 300, the rest arithmetic), the
// MMAs 670 from first to last.  Two rows of 3,500 .. 4,095 queries: 168 us, 1.0
// PFLOP/s; head_dim 256, whose pairs have twice the MMAs for the same sums: 111 us,
// 1.2 PFLOP/s (tensor 52 %).
//
// How (one persistent CTA per SM):
//  - Work is laid out along a line: for every (row, kv head) its blocks of keys,
//    for every block the steps through the query tiles that see it.  Every CTA
//    takes an equal range; it finds it itself from the row arrays (no plan
//    kernel, no host readback).  Rows whose queries fit one tile go by blocks of
//    128 keys, as runs; others by 256, so that the query tiles stream past two key
//    tiles at once; and those with few query tiles over a long context by 512 (head_dim
//    128 and 64), so that a block has steps enough: 8 rows of 64 queries on 8,192 tokens
//    take 48 us by 512 and 50 by 256, of 256 queries 129 and 137; past twelve steps
//    the two are even (448 queries 219 and 220, head_dim 64 211 and 209).  Where the
//    queries are the row 512 goes far past the causal limit: 64 prompts of 512 tokens
//    take 172 us by 512 and 127 by 256, 2 of 4,096 152 and 139.
//  - A block cut between CTAs leaves partial sums in the workspace; the last
//    CTA to arrive (a ticket for every 32 keys) adds them up in the order of the
//    line, so results do not depend on timing.
//  - Warps: 0 loads K; 2 cuts the range into runs, hands them out through a ring
//    and loads the query tiles; 1 and 3 issue the MMAs, every other pair each (one
//    warp for all took 180 us where two took 106, head_dim 256); 4-19 sum, four warps to a
//    pair, each group with an accumulator of its own.  The sums tell the loaders
//    what is free: as commits of the issuing warps that took 43 us for 41 (decode).
//  - The exponent is the difference d of score and lse, rounded once, and only
//    then in base 2: what the conversion rounds goes with d and not with the
//    score.  From the score on a weight is off by at most (3 |d| + 4) 2^-24 of
//    itself.  (Score and lse each in base 2 first, which saves a multiplication for
//    two weights and 3 to 5 % of the time of prompts, took a rounding of the whole
//    score into every weight: 3e-5 of it at scores of 200.)
//  - The score itself is the sum of exact products that the tensor cores make in
//    fp32: 16 at a time are added to what is there, and what does not fit is cut
//    off.  It falls short by 1.4e-7 of itself at head_dim 64, 2e-7 at 128 and 6e-7
//    at 256 (measured, scores near 20), and a weight by that much of the score:
//    3e-6, 4e-6 and 1.1e-5.  Scores around 0 leave weights within 3e-7 .. 6e-7.
//  - Sums of a step's columns are plain fp32 (four runs of 32 terms); steps are
//    added up with a compensation for what the addition drops, so thousands of
//    queries lose nothing.
#include <cuda_bf16.h>
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kMmKeysLog = 7;
constexpr int kMmKeys = 128;     // keys of a tile: M of every MMA
constexpr int kMmCols = 128;     // (query, head) columns of a query tile
constexpr int kMmFewSteps = 12;  // up to here, and with this many cached tokens to a step, a block
constexpr int kMmTokensPerStep = 256; // has four key tiles
constexpr int kFixCost = 2;      // positions that a key tile costs before its first step
constexpr int kMinRange = 6;     // positions that are worth a CTA of their own
constexpr int kMmMaxCtas = 160;  // persistent CTAs the workspace has room for
constexpr int kMmKWarp = 0, kMmMmaWarp = 1, kMmQWarp = 2, kMmMmaWarp2 = 3, kMmSumWarp = 4;
constexpr int kMmThreads = 640;
constexpr int kMmRuns = 8;       // runs of blocks handed out and not yet done with
constexpr int kMmReaders = 20;   // warps that read them
constexpr int kMmNoQuery = 0x7fffffff; // of a column that a query tile does not have
constexpr int kMmBadTiles = 16;  // key tiles whose bad pages are remembered

template <int D> struct MmCfg {
    static constexpr int kMostTiles = D == 256 ? 2 : 4;        // key tiles of a block
    static constexpr uint32_t kKBytes = kMmKeys * D * 2;
    static constexpr int kKStages = D == 64 ? 8 : D == 128 ? 4 : 2; // 128 KB
    static constexpr int kChunks = D / 64;                     // a query tile comes in chunks of 64 values
    static constexpr uint32_t kQBytes = kMmCols * 128;         // chunk: 128 rows of 128 B, swizzled
    static constexpr int kQStages = 5;
    static constexpr uint32_t kGroupStride = 8 * D * 2;        // 8 keys, all of head_dim
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffQ = kOffK + kKStages * kKBytes;
    static constexpr uint32_t kOffLse = kOffQ + kQStages * kQBytes; // [group of warps][three steps][128 columns]
    static constexpr uint32_t kOffHalf = kOffLse + 4 * 3 * 128 * 4; // [pair of groups][128 keys]
    static constexpr uint32_t kOffBar = kOffHalf + 2 * 128 * 4;
    static constexpr uint32_t kSmem = kOffBar + 2048;
    static constexpr uint32_t kTmemCols = 4 * kMmCols;         // an accumulator for each group of warps
    static_assert(kSmem <= 232448, "shared memory");
};

// What the roles need to know of a run: blocks of keys of one (row, kv head),
// one after the other.  More than one block only where each has one key tile
// and one step; a block with more steps is a run of its own.
struct MmRun {
    int32_t b, g;           // row, kv head
    int32_t tok, blocks;    // first key, blocks
    int32_t tiles;          // key tiles of a block: 1, 2 or 4; 0: no more runs
    int32_t first, queries; // the row's queries
    int32_t len, keys;      // cached tokens before the step, and with it
    int32_t step0, step1;   // steps of this piece: query tiles
    int32_t fresh, gone;
    int32_t piece0, pieces; // CTA of the block's first piece, pieces (1: whole)
};

struct MmRow {
    int first, queries, len, fresh, gone;
    int steps;  // of a block that all queries see
    int tiles;  // key tiles of a block
    int blocks; // of a kv head; 0: nothing to do
    int full;   // blocks, from the first on, that all query tiles see
    int err;
    int64_t work; // positions of a kv head
};

// a / b for a >= 0 and b > 0: nearly always small ones, whose division is a
// fraction of a 64-bit one.
__device__ __forceinline__ int64_t mm_div(int64_t a, int64_t b)
{
    return ((uint64_t)a | (uint64_t)b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The line cut into `ctas` ranges as equal as can be.
struct MmCut {
    int64_t quot;
    int rest, ctas;
    __device__ __forceinline__ int64_t lo(int c) const { return quot * c + rest * c / ctas; }
    // the CTA whose range holds position x
    __device__ __forceinline__ int of(int64_t x) const
    {
        int c = (int)min((int64_t)ctas - 1, mm_div(x, quot));
        while (lo(c) > x)
            --c;
        return c;
    }
};

// Where a CTA's range starts, and its length in positions.
struct MmStart {
    MmCut cut;
    int64_t at, off, left; // position on the line, within the (row, kv head), positions of the range
    int b, g;
    MmRow row;
};

struct MmBars {
    uint64_t k_full[8], k_empty[8];
    uint64_t q_full[5], q_empty[5];
    uint64_t s_full[4], s_free[4]; // [group of warps]
    uint64_t z_full[4];            // [group of warps]: its columns' lse are there
    uint64_t half_full[2], half_free[2]; // [pair of groups]: the one's sums for the other
    uint64_t run_full[kMmRuns], run_empty[kMmRuns];
    uint64_t drain;
    MmStart start;
    int64_t scratch[kMmThreads / 32];
    MmRun run[kMmRuns];
    uint16_t bad[kMmBadTiles]; // bit i: the page of a tile's keys 8 i .. 8 i + 7 is out of range
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(MmBars) <= 2048, "barrier block");

struct MmParams {
    const int32_t *indptr, *table, *seqlens, *fresh_from, *evicted;
    const float *lse;
    float *mass;
    int32_t *pos, *err_flag;
    int32_t *tickets; // [CTA][tile][quarter]: pieces of a block's 32 keys that are there
    float *parts;     // [CTA][begun before this CTA / in it][512 keys]
    float scale;      // softmax_scale
    int batch, num_q_heads, num_kv_heads, group, total_q, max_blocks;
    int page_shift, box_shift, num_pages, layout, slots;
    int q_tile;     // queries of a query tile
    int most_tiles; // key tiles of a block
    uint32_t q_box_bytes, q_one_bytes;
};

struct MmMaps {
    CUtensorMap k, q, q_one;
};

// ---------------------------------------------------------------- work line

__device__ __forceinline__ int mm_steps(const MmParams &p, const MmRow &r, int kb)
{
    const int i0 = kb * r.tiles * kMmKeys - r.len; // the block's first key is seen from this query on
    return r.steps - (i0 > 0 ? i0 / p.q_tile : 0);
}
__device__ __forceinline__ int64_t mm_cost(const MmRow &r, int steps)
{
    return (int64_t)r.tiles * (kFixCost + steps);
}

// What a row's part in the call is made from.
struct MmRaw {
    int first, end, len, fresh, gone;
};
__device__ __forceinline__ MmRaw mm_raw(const MmParams &p, int b)
{
    MmRaw raw;
    b = max(0, min(b, p.batch - 1));
    raw.first = p.indptr != nullptr ? p.indptr[b] : b;
    raw.end = p.indptr != nullptr ? p.indptr[b + 1] : b + 1;
    raw.len = p.seqlens[b];
    raw.fresh = p.fresh_from != nullptr ? p.fresh_from[b] : raw.len;
    raw.gone = p.evicted != nullptr ? p.evicted[b] : 0;
    return raw;
}

// A row's part in the call (see include/pkv.h).
__device__ __forceinline__ MmRow mm_row(const MmParams &p, const MmRaw &raw)
{
    MmRow r;
    r.first = raw.first;
    r.len = raw.len;
    r.fresh = raw.fresh;
    r.gone = raw.gone;
    const int64_t n = (int64_t)raw.end - raw.first;
    r.err = r.blocks = r.full = r.queries = r.steps = 0;
    r.tiles = 1;
    r.work = 0;
    if (r.first < 0 || n < 0 || n > (int64_t)p.total_q - r.first) {
        r.err = PKV_ERR_QLEN;
        return r;
    }
    if (n == 0 || r.len < 0)
        return r;
    const int64_t keys = (int64_t)r.len + n;
    if (keys > min(min((int64_t)p.max_blocks << p.page_shift, (int64_t)p.slots), (int64_t)kMassMaxKeys)) {
        r.err = PKV_ERR_OVERFLOW;
        return r;
    }
    r.queries = (int)n;
    r.steps = r.queries <= p.q_tile ? 1 : (r.queries + p.q_tile - 1) / p.q_tile;
    r.tiles = r.steps == 1                                                             ? 1
              : r.steps <= kMmFewSteps && r.len / r.steps >= kMmTokensPerStep ? p.most_tiles
                                                                              : 2;
    const int shift = kMmKeysLog + (r.tiles >> 1); // log2 of a block's keys
    r.blocks = (int)((keys + (1 << shift) - 1) >> shift);
    r.full = (int)min((int64_t)r.blocks, (((int64_t)r.len + p.q_tile - 1) >> shift) + 1);
    r.work = r.full * mm_cost(r, r.steps);
#pragma unroll 1
    for (int kb = r.full; kb < r.blocks; ++kb)
        r.work += mm_cost(r, mm_steps(p, r, kb));
    return r;
}

// Finds the CTA's range: a prefix sum over the rows' work.  The whole CTA.
__device__ MmStart mm_start(const MmParams &p, int64_t *scratch, MmStart *found)
{
    constexpr int kPer = (kMaxMassBatch + kMmThreads - 1) / kMmThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = min(kPer, (p.batch + kMmThreads - 1) / kMmThreads);
    MmRow row[kPer];
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * per + i;
        row[i].work = 0;
        if (i < per && b < p.batch) {
            row[i] = mm_row(p, mm_raw(p, b));
            if (blockIdx.x == 0)
                set_error(p.err_flag, row[i].err);
        }
        sum += row[i].work * p.num_kv_heads;
    }
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    if (lane == 31)
        scratch[warp] = x;
    if (tid == 0) { // an empty range, at row 0
        found->at = found->off = found->left = 0;
        found->b = found->g = 0;
        found->row = row[0];
    }
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kMmThreads / 32; ++w) {
        const int64_t v = scratch[w];
        x += w < warp ? v : 0;
        total += v;
    }
    x -= sum;
    const int c = blockIdx.x;
    MmCut cut;
    cut.ctas = total >= (int64_t)gridDim.x * kMinRange ? (int)gridDim.x : max(1, (int)total / kMinRange);
    cut.quot = mm_div(total, cut.ctas);
    cut.rest = (int)(total - cut.quot * cut.ctas);
    if (c < cut.ctas) {
        const int64_t lo = cut.lo(c), hi = cut.lo(c + 1);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t size = row[i].work * p.num_kv_heads, in_row = lo - x;
            if (hi > lo && in_row >= 0 && in_row < size) {
                MmStart at;
                at.cut = cut;
                at.at = lo;
                at.left = hi - lo;
                at.b = tid * per + i;
                at.g = (int)mm_div(in_row, row[i].work);
                at.off = in_row - at.g * row[i].work;
                at.row = row[i];
                *found = at;
            }
            x += size;
        }
    }
    __syncthreads();
    return *found;
}

// ---------------------------------------------------------------- waits

__device__ __noinline__ bool mm_wait_slow(uint64_t *bar, uint32_t parity, MmBars &bars, int32_t *err_flag)
{
    const uint64_t start = globaltimer_ns();
    volatile int32_t *abort = &bars.abort;
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity))
                return true;
        if (*abort != 0)
            return false;
        if (globaltimer_ns() - start > kWaitLimitNs) {
            *abort = 1;
            set_error(err_flag, PKV_ERR_TIMEOUT);
            return false;
        }
    }
}

// Bounded wait for the phase of the given parity; gives up when another role
// has.  A whole warp: all lanes get the same answer.  (Asking without being put to
// sleep takes issue slots from the sums: 2 to 15 % more time.)
__device__ __forceinline__ bool mm_wait(uint64_t *bar, uint32_t parity, MmBars &bars, int32_t *err_flag)
{
    bool done = mbar_try_wait(bar, parity);
    if (!done)
        done = mm_wait_slow(bar, parity, bars, err_flag);
    return __all_sync(0xffffffffu, done);
}

// ---------------------------------------------------------------- runs

// Cuts the CTA's range into runs, in order.  A whole warp.
struct MmWalk {
    MmCut cut;
    int64_t at, left, off; // position on the line, positions left, position within the block
    int b, g, kb;
    MmRow r;
    MmRaw then; // the next row, read ahead
    int n;      // runs handed out
    bool over;

    __device__ __forceinline__ void start(const MmParams &p, const MmStart &from)
    {
        cut = from.cut;
        at = from.at;
        left = from.left;
        off = from.off;
        b = from.b;
        g = from.g;
        kb = 0;
        r = from.row;
        then = mm_raw(p, b + 1);
        n = 0;
        over = false;
        if (left > 0) { // the block that the range starts in
            const int64_t size = mm_cost(r, r.steps);
            kb = (int)min((int64_t)r.full, mm_div(off, size));
            off -= kb * size;
#pragma unroll 1
            while (kb >= r.full && off >= mm_cost(r, mm_steps(p, r, kb)))
                off -= mm_cost(r, mm_steps(p, r, kb++));
        }
    }
    // Whether the next run has a slot that all readers are done with.
    __device__ __forceinline__ bool room(MmBars &bars) const
    {
        return n < kMmRuns ||
               __all_sync(0xffffffffu, mbar_test_wait(&bars.run_empty[n % kMmRuns], (uint32_t)(n / kMmRuns - 1) & 1));
    }
    // Hands the next run out.
    __device__ __forceinline__ void publish(const MmParams &p, MmBars &bars, int lane)
    {
        MmRun s;
        s.tiles = 0;
        while (left > 0) {
            if (kb >= r.blocks) {
                kb = 0;
                if (r.blocks == 0 || ++g == p.num_kv_heads) { // (positions are left: there is a next row)
                    g = 0;
                    ++b;
                    r = mm_row(p, then);
                    then = mm_raw(p, b + 1);
                }
                continue;
            }
            const int t = r.tiles;
            s.piece0 = blockIdx.x;
            s.pieces = 1;
            s.blocks = 1;
            int block = kb;
            if (r.steps == 1) { // blocks of one step: those whose step lies in the range
                constexpr int kSize = kFixCost + 1;
                const int64_t most = (int64_t)(r.blocks - kb) * kSize - off, take = min(most, left);
                const int first = off > kFixCost ? kb + 1 : kb;
                // positions from block kb's start; a step at or past them belongs to the next CTA
                const int end = (int)mm_div(off + take + kSize - 1 - kFixCost, kSize) + kb;
                left -= take;
                at += take;
                off += take;
                const int passed = (int)mm_div(off, kSize);
                kb += passed;
                off -= (int64_t)passed * kSize;
                if (first >= end)
                    continue;
                block = first;
                s.blocks = end - first;
                s.step0 = 0;
                s.step1 = 1;
            } else {
                const int steps = mm_steps(p, r, kb);
                const int64_t size = mm_cost(r, steps), take = min(size - off, left);
                const int shift = t >> 1; // log2 of t
                auto step_at = [&](int64_t x) { // first step whose position is x or more
                    return (int)max((int64_t)0, min((int64_t)steps, ((x + t - 1) >> shift) - kFixCost));
                };
                const int s0 = step_at(off), s1 = step_at(off + take);
                const int64_t start = at - off; // of the block
                at += take;
                left -= take;
                off += take;
                if (off >= size) {
                    off = 0;
                    ++kb;
                }
                if (s0 >= s1)
                    continue;
                s.step0 = r.steps - steps + s0;
                s.step1 = r.steps - steps + s1;
                if (s1 - s0 < steps) {
                    s.piece0 = cut.of(start + (int64_t)t * kFixCost);
                    s.pieces = cut.of(start + (int64_t)t * (kFixCost + steps - 1)) - s.piece0 + 1;
                }
            }
            s.b = b;
            s.g = g;
            s.tok = block * t * kMmKeys;
            s.tiles = t;
            s.first = r.first;
            s.queries = r.queries;
            s.len = r.len;
            s.keys = r.len + r.queries;
            s.fresh = r.fresh;
            s.gone = r.gone;
            break;
        }
        const int slot = n % kMmRuns;
        if (lane == 0) {
            bars.run[slot] = s;
            mbar_arrive(&bars.run_full[slot]);
        }
        ++n;
        over = s.tiles == 0;
    }
};

// The n-th run; a role that gave up sees the end.
__device__ __forceinline__ MmRun mm_run(const MmParams &p, MmBars &bars, int n)
{
    MmRun s;
    if (mm_wait(&bars.run_full[n % kMmRuns], (uint32_t)(n / kMmRuns) & 1, bars, p.err_flag))
        s = bars.run[n % kMmRuns];
    else
        s.tiles = 0;
    return s;
}
__device__ __forceinline__ void mm_run_done(MmBars &bars, int n, int lane)
{
    __syncwarp();
    if (lane == 0)
        mbar_arrive(&bars.run_empty[n % kMmRuns]);
}

// ---------------------------------------------------------------- loads

// One warp loads all key tiles, one box per lane: boxes of min(page, 64) keys, at
// most 16 a tile.  A page id outside the pool loads nothing and marks the tile.
template <int D>
__device__ void mm_load_k(const MmParams &p, const MmMaps &maps, uint8_t *smem, MmBars &bars, int lane)
{
    using C = MmCfg<D>;
    const int bsh = p.box_shift, boxes = kMmKeys >> bsh;
    const uint32_t box_bytes = (uint32_t)(1 << bsh) * D * 2;
    const bool nhd = p.layout == PKV_NHD;
    int n = 0, slot = 0, issued = 0;
    uint32_t round = 0; // times the ring has been filled
    MmRun s = mm_run(p, bars, 0);
    int tok = s.tok, end = s.tok + s.blocks * s.tiles * kMmKeys;
    auto page_of = [&](int at) { // this lane's page of the tile at `at`
        at += lane << bsh;
        return lane < boxes && at < s.keys ? p.table[(int64_t)s.b * p.max_blocks + (at >> p.page_shift)] : 0;
    };
    int id = s.tiles > 0 ? page_of(tok) : 0;
    while (s.tiles > 0) {
        const int at = tok + (lane << bsh), g = s.g, page = id;
        const bool want = lane < boxes && at < s.keys; // (of tiles behind the row's end, none)
        const bool good = want && page >= 1 && page < p.num_pages;
        // the page of the next tile, a tile ahead
        const int then = tok + kMmKeys;
        if (then >= end) {
            mm_run_done(bars, n, lane);
            s = mm_run(p, bars, ++n);
            tok = s.tok;
            end = s.tok + s.blocks * s.tiles * kMmKeys;
        } else {
            tok = then;
        }
        if (s.tiles > 0)
            id = page_of(tok);
        if (round > 0 && !mm_wait(&bars.k_empty[slot], (round - 1) & 1, bars, p.err_flag))
            break;
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, good));
        const uint32_t miss = __ballot_sync(0xffffffffu, want && !good);
        if (lane == 0) {
            uint32_t bits = 0; // a bit for 8 keys
            for (uint32_t m = miss; m != 0; m &= m - 1)
                bits |= ((1u << (1 << bsh >> 3)) - 1) << ((__ffs(m) - 1) << bsh >> 3);
            *(volatile uint16_t *)&bars.bad[issued % kMmBadTiles] = (uint16_t)bits;
            if (miss != 0)
                set_error(p.err_flag, PKV_ERR_PAGE);
            mbar_arrive_expect_tx(&bars.k_full[slot], count * box_bytes);
        }
        __syncwarp();
        if (good) {
            const int in_page = at & ((1 << p.page_shift) - 1);
            const int c3 = nhd ? ((page << p.page_shift) + in_page) >> 3 : in_page >> 3;
            const int c4 = nhd ? g : page * p.num_kv_heads + g;
            tma_load_5d_plain(smem + C::kOffK + slot * C::kKBytes + lane * box_bytes, &maps.k, 0, 0, 0, c3, c4,
                              &bars.k_full[slot]);
        }
        ++issued;
        if (++slot == C::kKStages) {
            slot = 0;
            ++round;
        }
    }
    // Copies still in flight (a role gave up): they land before the CTA ends.
    for (int k = issued > C::kKStages ? issued - C::kKStages : 0; k < issued; ++k)
        mbar_wait(&bars.k_full[k % C::kKStages], (uint32_t)(k / C::kKStages) & 1);
}

// One warp cuts the range into runs and loads the query tiles of every step, a box
// per 64 columns.  It hands runs out ahead of what it loads itself, two a step,
// so that the key tiles of the next runs are on their way.
template <int D>
__device__ void mm_load_q(const MmParams &p, const MmMaps &maps, uint8_t *smem, MmBars &bars, const MmStart &from, int lane)
{
    using C = MmCfg<D>;
    MmWalk walk;
    walk.start(p, from);
    walk.publish(p, bars, lane);
    int slot = 0, issued = 0;
    uint32_t round = 0;
    bool going = true;
    for (int n = 0; going; ++n) {
        while (!walk.over && walk.n <= n) {
            if (!walk.room(bars) && !mm_wait(&bars.run_empty[walk.n % kMmRuns], (uint32_t)(walk.n / kMmRuns - 1) & 1, bars,
                                             p.err_flag)) {
                going = false;
                break;
            }
            walk.publish(p, bars, lane);
        }
        const MmRun s = mm_run(p, bars, n);
        if (s.tiles == 0)
            break;
        const bool one = s.queries == 1; // a box of one query: no other row's are fetched
        const uint32_t bytes = one ? p.q_one_bytes : p.q_box_bytes;
        for (int st = s.step0; st < s.step1 && going; ++st) {
            for (int c = 0; c < C::kChunks; ++c) {
                if (round > 0 && !mm_wait(&bars.q_empty[slot], (round - 1) & 1, bars, p.err_flag)) {
                    going = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars.q_full[slot], bytes);
                    tma_load_3d_plain(smem + C::kOffQ + slot * C::kQBytes, one ? &maps.q_one : &maps.q, c * 64,
                                      s.g * p.group, s.first + st * p.q_tile, &bars.q_full[slot]);
                }
                __syncwarp();
                ++issued;
                if (++slot == C::kQStages) {
                    slot = 0;
                    ++round;
                }
            }
            for (int k = 0; k < 2 && !walk.over && walk.room(bars); ++k)
                walk.publish(p, bars, lane);
        }
        mm_run_done(bars, n, lane);
    }
    for (int k = issued > C::kQStages ? issued - C::kQStages : 0; k < issued; ++k)
        mbar_wait(&bars.q_full[k % C::kQStages], (uint32_t)(k / C::kQStages) & 1);
}

// ---------------------------------------------------------------- MMA

// Four MMAs of 64 values of the inner dimension: A and B 32 bytes on each time.
// The whole warp; one elected thread (always the same) issues.
__device__ __forceinline__ void mm_mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred e, p, t;\n\t"
                 ".reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.eq.b32 t, 0, 0;\n\t"
                 "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
                 "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void mm_commit(uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                     smem_addr(bar))
                 : "memory");
}

// One arrival of the warp.
__device__ __forceinline__ void mm_arrive(uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar))
                 : "memory");
}

// Two warps issue, every other (key tile, step) pair each (`half`: which), and so
// have two accumulators and every other key slot to themselves: what a pair costs
// a warp besides its MMAs (waits, votes, descriptors: 500 cycles) then overlaps
// the other warp's.
template <int D>
__device__ void mm_mma(const MmParams &p, uint8_t *smem, MmBars &bars, uint32_t tmem, uint32_t half, int lane)
{
    using C = MmCfg<D>;
    constexpr int kChunks = C::kChunks;
    const uint64_t kd0 = tc_sw128_desc(smem_addr(smem + C::kOffK), 16, C::kGroupStride);
    const uint64_t qd0 = tc_sw128_desc(smem_addr(smem + C::kOffQ), 16, 1024);
    uint32_t tile0 = 0, seq = 0; // key tiles, pairs before the block (alike modulo 2)
    uint32_t q_slot = 0, q_par = 0; // of the next chunk
    bool going = true;
    for (int n = 0; going; ++n) {
        const MmRun s = mm_run(p, bars, n);
        // warp-uniform values (read from one lane) stay in uniform registers
        const int tiles = __shfl_sync(0xffffffffu, s.tiles, 0);
        if (tiles == 0)
            break;
        const int step0 = __shfl_sync(0xffffffffu, s.step0, 0), step1 = __shfl_sync(0xffffffffu, s.step1, 0);
        const int queries = __shfl_sync(0xffffffffu, s.queries, 0), blocks = __shfl_sync(0xffffffffu, s.blocks, 0);
        // key tiles of the run that lie before the row's end
        const int real = __shfl_sync(0xffffffffu, (s.keys - s.tok + kMmKeys - 1) / kMmKeys, 0);
        mm_run_done(bars, n, lane);
        // the accumulator of pair u, and the key tile x if it is new, are there
        auto ready = [&](uint32_t u, uint32_t x, bool new_k) {
            return (!new_k || mm_wait(&bars.k_full[x % C::kKStages], x / C::kKStages & 1, bars, p.err_flag)) &&
                   (u < 4 || mm_wait(&bars.s_free[u & 3], ((u >> 2) - 1) & 1, bars, p.err_flag));
        };
        auto k_desc = [&](uint32_t x) { return kd0 + (uint64_t)(x % C::kKStages * C::kKBytes >> 4); };
#pragma unroll 1
        for (int st = step0; st < step1 && going; ++st) {
            const int cols = (min(p.q_tile, queries - st * p.q_tile) * p.group + 15) & ~15;
            const uint32_t idesc = tc_idesc_bf16(kMmKeys, 0, false, false) | (uint32_t)(cols >> 3) << 17;
            uint64_t qd[kChunks]; // of the step's chunks
            const bool by_chunk = kChunks > 2 && tiles > 1;
            // (every phase of these barriers is waited for, with pairs to issue or not)
            auto next_chunk = [&](int c) {
                if (!mm_wait(&bars.q_full[q_slot], q_par, bars, p.err_flag))
                    going = false;
                qd[c] = qd0 + (uint64_t)(q_slot * C::kQBytes >> 4);
                const uint32_t slot = q_slot;
                if (++q_slot == C::kQStages) {
                    q_slot = 0;
                    q_par ^= 1;
                }
                return slot;
            };
            if (!by_chunk) { // all chunks, then the key tiles (or the run's blocks) one by one
                const int pairs = tiles == 1 ? blocks : tiles;
                // For a single pair the other warp issues nothing, and the sums' arrival says
                // nothing of its wait: without an arrival of its own a chunk could be loaded
                // over, and its barrier two phases on, before this warp has looked.
                const bool idle = pairs == 1 && ((half ^ seq) & 1) != 0;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const uint32_t slot = next_chunk(c);
                    if (idle)
                        mm_arrive(&bars.q_empty[slot]);
                }
#pragma unroll 1
                for (int j = (half ^ seq) & 1; j < pairs && going; j += 2) {
                    const uint32_t u = seq + j, x = tile0 + j;
                    if (!ready(u, x, st == step0)) {
                        going = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t kd = k_desc(x);
                    const uint32_t d = tmem + (u & 3) * kMmCols;
                    if (j < real) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c)
                            mm_mma4(d, kd + (uint64_t)(c * 1024 >> 4), qd[c], idesc, c > 0 ? 1u : 0u);
                    }
                    mm_commit(&bars.s_full[u & 3]);
                }
                seq += pairs;
            } else { // head_dim 256: a query tile nearly fills the ring, so its chunks are freed one by one
                const int j = (half ^ seq) & 1; // (two key tiles)
                const uint32_t u = seq + j, x = tile0 + j;
                const uint64_t kd = k_desc(x);
#pragma unroll 1
                for (int c = 0; c < kChunks && going; ++c) {
                    const uint32_t slot = next_chunk(0);
                    if (!going || (c == 0 && !ready(u, x, st == step0))) {
                        going = false;
                        break;
                    }
                    tc_fence_after();
                    if (j < real)
                        mm_mma4(tmem + (u & 3) * kMmCols, kd + (uint64_t)(c * 1024 >> 4), qd[0], idesc, c > 0 ? 1u : 0u);
                    mm_commit(&bars.q_empty[slot]);
                }
                mm_commit(&bars.s_full[u & 3]);
                seq += tiles;
            }
        }
        tile0 += tiles * blocks;
    }
    mm_commit(&bars.drain); // the commits have arrived before the CTA ends
    mbar_wait(&bars.drain, 0);
}

// ---------------------------------------------------------------- sums

// 32 (16) consecutive columns of this thread's lane, waited for.  (With the wait
// apart from the load, so that sums could go on meanwhile, every value was moved
// once more between the two.)
#define PKV_O8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                  "=r"(r[i + 6]), "=r"(r[i + 7])
__device__ __forceinline__ void mm_ld(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : PKV_O8(0), PKV_O8(8), PKV_O8(16), PKV_O8(24)
                 : "r"(taddr));
}
__device__ __forceinline__ void mm_ld(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : PKV_O8(0), PKV_O8(8)
                 : "r"(taddr));
}
#undef PKV_O8

// The sum of e^(x scale + z) over N columns; z holds -lse.
template <bool MASKED, int N>
__device__ __forceinline__ void mm_sum_of(const uint32_t (&x)[N], const float *z, float scale, int from, int to,
                                          float2 &sum0, float2 &sum1)
{
    const float2 s2 = make_float2(scale, scale), log2e = make_float2(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 z4 = *reinterpret_cast<const float4 *>(z + i);
        const float2 a = fmul2(ffma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), s2,
                                     make_float2(z4.x, z4.y)), log2e);
        const float2 c = fmul2(ffma2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), s2,
                                     make_float2(z4.z, z4.w)), log2e);
        float2 w0 = make_float2(ex2_approx(a.x), ex2_approx(a.y));
        float2 w1 = make_float2(ex2_approx(c.x), ex2_approx(c.y));
        if (MASKED) {
            w0.x = i >= from && i < to ? w0.x : 0.f;
            w0.y = i + 1 >= from && i + 1 < to ? w0.y : 0.f;
            w1.x = i + 2 >= from && i + 2 < to ? w1.x : 0.f;
            w1.y = i + 3 >= from && i + 3 < to ? w1.y : 0.f;
        }
        sum0 = __fadd2_rn(sum0, w0);
        sum1 = __fadd2_rn(sum1, w1);
    }
}

// Adds one to a ticket, ordering this warp's stores before it and the other
// pieces' stores before what follows.
__device__ __forceinline__ int mm_ticket(int32_t *ticket)
{
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(ticket) : "memory");
    return old;
}

// Adds y to a sum, with what earlier additions dropped.
__device__ __forceinline__ void mm_add(float &sum, float &dropped, float y)
{
    y += dropped;
    const float next = sum + y;
    dropped = fabsf(next) < INFINITY ? y - (next - sum) : 0.f;
    sum = next;
}

template <int D>
__device__ void mm_sum(const MmParams &p, uint8_t *smem, MmBars &bars, uint32_t tmem, int warp, int lane)
{
    using C = MmCfg<D>;
    // Group w takes every fourth (key tile, step) pair of the CTA: of a block of
    // four key tiles one of them, of two every other step of one.
    const int w = (warp - kMmSumWarp) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + w * kMmCols;
    float *lse = reinterpret_cast<float *>(smem + C::kOffLse) + w * 384;
    float *half = reinterpret_cast<float *>(smem + C::kOffHalf) + (w & 1) * 128;
    // the (query, head) of this thread's column, whose lse it fetches for the group
    const int my_query = r / p.group < p.q_tile ? r / p.group : kMmNoQuery, my_head = r % p.group;
    int room = 256; // where the lse written last are
    uint32_t tile0 = 0;
    uint32_t q0 = 0; // chunks of query tiles before the run
    uint32_t seq = 0, taken = 0, staged = 0, halves = 0; // pairs before the run, taken by the group; lse; shared blocks
    for (int n = 0;; ++n) {
        const MmRun s = mm_run(p, bars, n);
        if (s.tiles == 0)
            return;
        const int steps = s.step1 - s.step0, rank = (w - seq) & 3;
        // tile within the block, first step and block of this group's, the way to the next
        const int j = s.tiles == 4 ? rank : s.tiles == 2 ? rank & 1 : 0;
        int st = s.step0 + (s.tiles == 2 ? rank >> 1 : 0), blk = s.tiles == 1 ? rank : 0;
        const int next_step = s.tiles == 4 ? 1 : 2;
        const bool shared = s.tiles == 2 && steps > 1; // with the group that has the other steps
        const bool ends = !shared || ((s.step1 - st) & 1) != 0; // this group finishes the block
        // The columns' lse go through shared memory, a step ahead: while step k is
        // summed those of k + 1 are written and those of k + 2 are on their way.
        const float *z_at = p.lse + ((int64_t)s.first + (my_query == kMmNoQuery ? 0 : my_query)) * p.num_q_heads +
                            s.g * p.group + my_head;
        auto fetch = [&](int step) {
            const int q = step * p.q_tile;
            return step < s.step1 && my_query < s.queries - q ? z_at[(int64_t)q * p.num_q_heads] : 0.f;
        };
        auto stage = [&](float z) {
            room = room == 256 ? 0 : room + 128;
            lse[room + r] = z == -INFINITY ? z : -z;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars.z_full[w]);
            ++staged;
        };
        float z = 0.f;
        if (st < s.step1 && blk < s.blocks) {
            const float first = fetch(st);
            z = s.tiles > 1 ? fetch(st + next_step) : 0.f;
            stage(first);
        }
        float sum = 0.f, dropped = 0.f, was = 0.f;
        const int64_t unit = ((int64_t)s.b * p.num_kv_heads + s.g) * p.slots;
        const int whole_steps = p.q_tile * p.group == kMmCols ? s.queries / p.q_tile : 0; // with all columns
        const float *zs = lse;
        int tok = 0, key = 0;
        bool fresh = false, mine = false, new_z = true, begins = true;
#pragma unroll 1
        while (st < s.step1 && blk < s.blocks) {
            if (begins) {
                tok = s.tok + (blk * s.tiles + j) * kMmKeys;
                key = tok + r;
                fresh = key >= s.fresh;
                mine = ends && key < s.keys;
                sum = dropped = was = 0.f;
                if (mine && !fresh)
                    was = p.mass[unit + key];
            }
            if (new_z) {
                if (!mm_wait(&bars.z_full[w], (staged - 1) & 1, bars, p.err_flag))
                    return;
                zs = lse + room;
            }
            const int now = st;
            if (s.tiles == 1) {
                blk += 4;
                new_z = false;
            } else {
                begins = false;
                st += next_step;
                if (st < s.step1) {
                    // (the room was last read three steps ago: all of the group have staged since)
                    stage(z);
                    z = fetch(st + next_step);
                }
            }
            if (!mm_wait(&bars.s_full[w], taken & 1, bars, p.err_flag))
                return;
            ++taken;
            // What the MMAs have read is free: the key tile after its last step, the
            // query tile after the last pairs of the two issuing warps (of a single pair
            // the other warp tells itself).  (Told from here: a commit for it would cost
            // those warps more than an MMA does.)
            const uint32_t tile = tile0 + (uint32_t)(tok - s.tok) / kMmKeys;
            if (quarter == 0 && lane == 0) {
                if (now == s.step1 - 1)
                    mbar_arrive(&bars.k_empty[tile % C::kKStages]);
                const int pairs = s.tiles == 1 ? s.blocks : s.tiles, pair = s.tiles == 1 ? blk - 4 : j;
                if ((C::kChunks <= 2 || s.tiles == 1) && pair >= pairs - 2)
#pragma unroll
                    for (int c = 0; c < C::kChunks; ++c)
                        mbar_arrive(&bars.q_empty[(q0 + (now - s.step0) * C::kChunks + c) % C::kQStages]);
            }
            tc_fence_after();
            auto leave = [&] { // all of the accumulator is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.s_free[w]);
            };
            float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
            const int start = now * p.q_tile;                    // query of the first column
            const bool edge = tok + kMmKeys - 1 - s.len > start; // some queries do not see all of the tile
            if (now < whole_steps && !edge && tok < s.keys) {    // all columns
#pragma unroll
                for (int c = 0; c < kMmCols; c += 32) {
                    uint32_t x[32];
                    mm_ld(acc + c, x);
                    if (c + 32 == kMmCols)
                        leave();
                    mm_sum_of<false>(x, zs + c, p.scale, 0, 32, sum0, sum1);
                }
            } else {
                // columns of queries before the key's own see nothing of it; of a tile
                // behind the row's end there is nothing to sum
                const int seen = max(0, key - s.len - start) * p.group;
                const int cols = tok < s.keys ? min(p.q_tile, s.queries - start) * p.group : 0;
                const int whole = edge ? 0 : cols & ~15;
                uint32_t x[16];
                if (cols == 0)
                    leave();
#pragma unroll 1
                for (int c = 0; c < whole; c += 16) {
                    mm_ld(acc + c, x);
                    if (c + 16 >= cols)
                        leave();
                    mm_sum_of<false>(x, zs + c, p.scale, 0, 16, sum0, sum1);
                }
#pragma unroll 1
                for (int c = whole; c < cols; c += 16) {
                    mm_ld(acc + c, x);
                    if (c + 16 >= cols)
                        leave();
                    mm_sum_of<true>(x, zs + c, p.scale, seen - c, cols - c, sum0, sum1);
                }
            }
            mm_add(sum, dropped, (sum0.x + sum1.x) + (sum0.y + sum1.y));
            if (s.tiles > 1 && st < s.step1)
                continue;
            // the block's sums
            if (shared) {
                if (!ends) {
                    if (halves > 0 && !mm_wait(&bars.half_free[w & 1], (halves - 1) & 1, bars, p.err_flag))
                        return;
                    half[r] = sum;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bars.half_full[w & 1]);
                } else {
                    if (!mm_wait(&bars.half_full[w & 1], halves & 1, bars, p.err_flag))
                        return;
                    mm_add(sum, dropped, half[r]);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bars.half_free[w & 1]);
                }
            }
            bool last = ends;
            if (ends && s.pieces > 1) {
                float *slot = p.parts + j * kMmKeys + r;
                __stcg(slot + (2 * blockIdx.x + (s.piece0 == blockIdx.x ? 1 : 0)) * 512, sum);
                int32_t *ticket = p.tickets + (s.piece0 * 4 + j) * 4 + quarter;
                __syncwarp();
                int old = 0;
                if (lane == 0)
                    old = mm_ticket(ticket);
                last = __shfl_sync(0xffffffffu, old, 0) == s.pieces - 1;
                __syncwarp();
                if (last) {
                    if (lane == 0)
                        *ticket = 0;
                    sum = __ldcg(slot + (2 * s.piece0 + 1) * 512);
                    dropped = 0.f;
                    for (int c = 1; c < s.pieces; ++c)
                        mm_add(sum, dropped, __ldcg(slot + 2 * (s.piece0 + c) * 512));
                }
            }
            const bool bad = (*(volatile uint16_t *)&bars.bad[tile % kMmBadTiles] >> (r >> 3)) & 1;
            if (last && mine && !bad) {
                p.mass[unit + key] = was + sum;
                if (fresh && p.pos != nullptr)
                    p.pos[unit + key] = key + s.gone;
            }
        }
        halves += shared ? 1 : 0;
        seq += (uint32_t)(s.tiles * steps * s.blocks);
        tile0 += s.blocks * s.tiles;
        q0 = (q0 + steps * C::kChunks) % C::kQStages;
        mm_run_done(bars, n, lane);
    }
}

// ---------------------------------------------------------------- kernel

template <int D>
__global__ void __launch_bounds__(kMmThreads, 1)
    mass_kernel(const __grid_constant__ MmParams p, const __grid_constant__ MmMaps maps)
{
    using C = MmCfg<D>;
    extern __shared__ __align__(1024) unsigned char mm_smem[];
    uint8_t *smem = mm_smem;
    if ((smem_addr(smem) & 1023u) != 0) { // the swizzled tiles need it; dynamic shared memory starts so
        set_error(p.err_flag, PKV_ERR_TIMEOUT);
        return;
    }
    MmBars &bars = *reinterpret_cast<MmBars *>(smem + C::kOffBar);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kKStages; ++i) {
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.k_empty[i], 1);
        }
        for (int i = 0; i < C::kQStages; ++i) {
            mbar_init(&bars.q_full[i], 1);
            mbar_init(&bars.q_empty[i], 2); // once for each issuing warp
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.s_free[i], 4);
            mbar_init(&bars.z_full[i], 4);
        }
        for (int i = 0; i < kMmRuns; ++i) {
            mbar_init(&bars.run_full[i], 1);
            mbar_init(&bars.run_empty[i], kMmReaders);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.half_full[i], 4);
            mbar_init(&bars.half_free[i], 4);
        }
        mbar_init(&bars.drain, 2);
        bars.abort = 0;
        mbar_init_fence();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.q_one);
    }
    const MmStart from = mm_start(p, bars.scratch, &bars.start);
    // TMEM while the first loads are on their way: those who load have no use for it.
    uint32_t tmem = 0;
    if (warp != kMmKWarp && warp != kMmQWarp) {
        if (warp == kMmMmaWarp) {
            tmem_alloc(&bars.tmem_base, C::kTmemCols);
            tmem_relinquish();
        }
        tc_fence_before();
        named_sync(1, kMmThreads - 64);
        tc_fence_after();
        tmem = __shfl_sync(0xffffffffu, bars.tmem_base, 0);
    }
    if (warp == kMmKWarp)
        mm_load_k<D>(p, maps, smem, bars, lane);
    else if (warp == kMmQWarp)
        mm_load_q<D>(p, maps, smem, bars, from, lane);
    else if (warp == kMmMmaWarp || warp == kMmMmaWarp2)
        mm_mma<D>(p, smem, bars, tmem, warp == kMmMmaWarp2 ? 1 : 0, lane);
    else
        mm_sum<D>(p, smem, bars, tmem, warp, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmMmaWarp)
        tmem_dealloc(tmem, C::kTmemCols);
}

// ---------------------------------------------------------------- host side

struct MmEntry {
    int D, most_tiles;
    const void *kernel;
    uint32_t smem;
};

const MmEntry kMmTable[] = {
    {64, MmCfg<64>::kMostTiles, reinterpret_cast<const void *>(&mass_kernel<64>), MmCfg<64>::kSmem},
    {128, MmCfg<128>::kMostTiles, reinterpret_cast<const void *>(&mass_kernel<128>), MmCfg<128>::kSmem},
    {256, MmCfg<256>::kMostTiles, reinterpret_cast<const void *>(&mass_kernel<256>), MmCfg<256>::kSmem},
};

const MmEntry *mm_find(int D)
{
    for (const MmEntry &e : kMmTable)
        if (e.D == D)
            return &e;
    return nullptr;
}

// Once per device: the kernel's shared memory.
bool mm_ready(int device, const MmEntry *e)
{
    constexpr int kDevices = 64;
    static bool done[kDevices][3] = {};
    if (device < 0 || device >= kDevices)
        return false;
    bool &slot = done[device][e - kMmTable];
    if (!slot)
        slot = cudaFuncSetAttribute(e->kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)e->smem) == cudaSuccess;
    return slot;
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

} // namespace

pkv_status mass_shape(int batch, int total_q, int max_blocks, int num_q_heads, const pkv_cache_desc *desc,
                      MassShape *s)
{
    const pkv_status st = check_desc(desc);
    if (st != PKV_OK)
        return st;
    if (batch < 0 || total_q < 0 || max_blocks < 1 || num_q_heads < 1 || num_q_heads % desc->num_kv_heads != 0)
        return PKV_EINVAL;
    s->group = num_q_heads / desc->num_kv_heads;
    if (batch > kMaxMassBatch || desc->page_size < 8 || s->group > kMmCols ||
        (int64_t)total_q * num_q_heads >= ((int64_t)1 << 31))
        return PKV_EUNSUPPORTED;
    s->q_tile = kMmCols / s->group;
    s->off_parts = kMmMaxCtas * 16 * sizeof(int32_t);
    s->bytes = 256 + s->off_parts + (size_t)kMmMaxCtas * 2 * 512 * sizeof(float);
    return PKV_OK;
}

} // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_mass_workspace_size(int32_t batch, int32_t total_q, int32_t max_blocks, int32_t num_q_heads,
                               const pkv_cache_desc *desc)
{
    MassShape s;
    return mass_shape(batch, total_q, max_blocks, num_q_heads, desc, &s) == PKV_OK ? s.bytes : 0;
}

pkv_status pkv_attn_mass(const pkv_cache_desc *desc, const void *k_cache, const void *q, const int32_t *qo_indptr,
                         const float *lse, const int32_t *block_table, int32_t max_blocks,
                         const int32_t *cache_seqlens, int32_t batch, int32_t num_q_heads, int32_t total_q,
                         float softmax_scale, const int32_t *fresh_from, const int32_t *evicted, float *mass,
                         int32_t *slot_pos, int32_t slots, void *workspace, size_t workspace_bytes, int32_t *err_flag,
                         void *stream)
{
    MassShape shape;
    const pkv_status st = mass_shape(batch, total_q, max_blocks, num_q_heads, desc, &shape);
    if (st != PKV_OK)
        return st;
    if (!isfinite(softmax_scale) || slots < 1 || (qo_indptr == nullptr && total_q != batch))
        return PKV_EINVAL;
    if (batch == 0 || total_q == 0)
        return PKV_OK;
    if (k_cache == nullptr || q == nullptr || lse == nullptr || block_table == nullptr || cache_seqlens == nullptr ||
        mass == nullptr || !aligned16(k_cache) || !aligned16(q) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
        !slots_aligned(mass, slots) || !slots_aligned(slot_pos, slots))
        return PKV_EINVAL;
    if (workspace == nullptr || workspace_bytes < shape.bytes || !aligned16(workspace))
        return PKV_EWORKSPACE;
    const MmEntry *e = mm_find(desc->head_dim);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !mm_ready(dev, e))
        return PKV_ECUDA;
    unsigned char *ws =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
    MmParams p;
    p.indptr = qo_indptr;
    p.table = block_table;
    p.seqlens = cache_seqlens;
    p.fresh_from = fresh_from;
    p.evicted = evicted;
    p.lse = lse;
    p.mass = mass;
    p.pos = slot_pos;
    p.err_flag = err_flag;
    p.tickets = reinterpret_cast<int32_t *>(ws);
    p.parts = reinterpret_cast<float *>(ws + shape.off_parts);
    p.scale = softmax_scale;
    p.batch = batch;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = desc->num_kv_heads;
    p.group = shape.group;
    p.total_q = total_q;
    p.max_blocks = max_blocks;
    p.page_shift = 0;
    while ((1 << p.page_shift) < desc->page_size)
        ++p.page_shift;
    p.box_shift = p.page_shift < 6 ? p.page_shift : 6;
    p.num_pages = desc->num_pages;
    p.layout = desc->layout;
    p.slots = slots;
    p.q_tile = shape.q_tile;
    p.most_tiles = e->most_tiles;
    const int box_q = shape.q_tile < total_q ? shape.q_tile : total_q;
    p.q_box_bytes = (uint32_t)box_q * shape.group * 128;
    p.q_one_bytes = (uint32_t)shape.group * 128;
    MmMaps m;
    if (encode_group_map(&m.k, *desc, const_cast<void *>(k_cache), 1 << p.box_shift) != CUDA_SUCCESS ||
        encode_q_map(&m.q, q, desc->head_dim, num_q_heads, total_q, shape.group, box_q) != CUDA_SUCCESS ||
        encode_q_map(&m.q_one, q, desc->head_dim, num_q_heads, total_q, shape.group, 1) != CUDA_SUCCESS)
        return PKV_ECUDA;
    const int grid = sm_count(dev) < kMmMaxCtas ? sm_count(dev) : kMmMaxCtas;
    void *args[] = {&p, &m};
    return cudaLaunchKernel(e->kernel, dim3(grid), dim3(kMmThreads), args, e->smem, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ECUDA;
}

} // extern "C"
