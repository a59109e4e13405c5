// pkv_tree_attn.cu -- attention of a tree of drafted tokens over the paged
// cache, on the 5th-generation tensor cores (tcgen05, TMEM accumulators).
//
// What it computes.  Node i of row b attends the row's L_b cached keys and
// drafted key j (position L_b + j) iff bit j of its mask is set
// (include/pkv.h): S = Q K^T, p = exp2(S scale log2(e) - m), O = p V / sum p.
//
// What bounds it.  A unit is (row, kv head, up to 128 (node, head) pairs): one
// MMA row tile, so a K/V byte is read once for all of them.  Per 128 keys at
// head_dim 128 a unit reads 64 KB, 1.45 us of an SM's share of the measured HBM
// rate, and needs 24 MMAs of 128 x 128 x 16 (8 for S, 16 for P V, whose P is
// kept as two bf16 parts), 0.8 us at the tensor peak: memory bounds it up to 128
// pairs whatever their number, the tensor pipe beyond (two row tiles read the
// same K/V from L2).  Measured (stamps of the SM clock): a step takes 1.3 us.
// With one row tile it waits for K, so memory it is; with more the MMA warp is
// busy throughout (S 0.25, P V 0.53, the rest its waits, commits and the walk:
// 0.1 us more in it is 0.1 us more a step, in the softmax half of that).  64
// uneven rows of two tiles, 64 nodes x 4 heads, take 148 us = 615 TFLOP/s, the
// tensor pipe active 54 % of the cycles (168 us with an election for every MMA
// and a row's tiles in one CTA, 157 with one for four MMAs, 149 with the tiles
// side by side, 147 with one barrier for P and V).  Short calls are bound by
// latency: 32 rows of 512 .. 1024 tokens with trees of 16 nodes take 37 us, 3.0
// TB/s, of which the start of the CTAs is 4, the append 3, the tail and the
// combine kernel 6; one node over 64 tokens takes 11.8 us for its three kernels.
//
// The roles' code is kept short (one walk of the range, loops not unrolled
// beyond 32 columns): at 120 KB a sixth of the instruction fetches missed the
// SM's instruction cache and a tile took half again as long.
//
// How (one persistent CTA per SM):
//  - The units are laid end to end as a line of positions (kStartCost for the
//    fixed cost of a unit, then its 64-token blocks) and every CTA takes an
//    equal range, so a long row is shared by many CTAs.  Each CTA finds its
//    range itself from the row arrays: no plan kernel, no host readback.
//    Where rows may have more nodes than a tile holds, two CTAs go along the line
//    side by side, one on the even, one on the odd units of a row: of a row of
//    two tiles they read the same K/V at the same time, so HBM delivers it once.
//    With the tiles one after the other in a CTA, long rows' K/V have left the L2
//    in between: 64 uneven rows of two tiles took 157 us for 149 and read 805 MB
//    from HBM for 465.  It takes an even number of units in every row, whatever
//    its tiles, and so an even number of kv heads; with an odd one the tiles go
//    one after the other, and rows of four tiles go as two such pairs (neither
//    has been measured).
//  - A unit inside one CTA's range is finished there.  The others leave (ref, l)
//    and O in the workspace, fp32, and a second kernel joins them in range
//    order (results do not depend on timing).  A CTA has at most two such
//    slices: the one it starts in and the one it ends in.
//  - Warps: 3 walks the CTA's range, hands its slices to the others through a
//    ring and looks V through; 0 loads Q and K, 2 loads V, with TMA, K and V into
//    a ring each (one lane per box, a box per page piece); 1 owns TMEM and one
//    thread of it issues the MMAs; 4-7 and 8-11 run the softmax, two threads per
//    MMA row on half of a tile's columns each (they exchange their maxima); 12-15
//    finish slices, so that the softmax goes on with the next one meanwhile.
//    While the softmax is at tile t the tensor pipe runs S of tile t + 1 and P V
//    of tile t - 1.
//  - The running maximum m moves only when a score exceeds it by more than 8, a
//    factor 2^8 (then O is rescaled).  The weights are taken as 2^(s - ref), ref = m + 8 +
//    slack with slack = 1 + ceil(log2 of the row's keys): none is above
//    2^-slack and they sum to at most 1/2, so values at the end of bf16 cannot
//    overflow O before the division.  What that costs is at the other end:
//    weights below 2^(slack - 118) of the row's largest, and values below about
//    that, are lost (slack is 17 at 64K keys).
//  - P replaces S in TMEM as bf16 hi + lo parts (16 significant bits; 8 alone
//    leave errors of 2^-9 of the row's scale in small outputs).
//  - Tiles with drafted keys take their visibility as 32-bit words, shifted
//    out of the node's mask.  V of drafted tokens is looked through in shared
//    memory before the MMAs read it: an infinity or NaN there is replaced by 0
//    for the MMA (0 * inf would reach nodes that do not see it) and added in
//    the epilogue to the nodes that do.  Cached tokens are seen by all: there
//    the finishing warps look at O, and where it is not finite they put the sum
//    of the values that are not (ta_mend_cached).  The look costs 0.4 us of one
//    node's 11.8, 0.8 of 37 and 1.6 of 148.
//  - Cutting the line: kStartCost 1 .. 4 and kMinRange 4 .. 16 were measured on
//    short, long, even and uneven batches: nothing better than 2 and 6 (a
//    minimum that grows with the rows in use: head_dim 256 43 -> 55 us).
#include <cuda_bf16.h>
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kTaRows = 128;      // M of every MMA
constexpr int kTaBlock = 64;      // tokens per position of the work line
constexpr int kStartCost = 2;     // positions that a unit costs before its first block
constexpr int kMinBlocks = 2;     // a unit is not cut nearer than this to its ends
constexpr int kMinRange = 6;      // positions that are worth a CTA of their own
constexpr int kTaMaxCtas = 160;   // persistent CTAs the workspace has room for
constexpr int kTaKWarp = 0, kTaMmaWarp = 1, kTaVWarp = 2, kTaWalkWarp = 3, kTaSoftmaxWarp = 4,
              kTaEndWarp = 12;
constexpr int kTaThreads = 512;
constexpr int kSlices = 8;        // slices handed out and not yet done with
constexpr int kReaders = 16;      // warps that read them
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLn2 = 0.693147180559945309f;

// Record of a CTA's shared slices (combine kernel).
constexpr int kHeadValid = 1, kHeadEnd = 2, kTail = 4, kHeadBad = 8, kTailBad = 16;

template <int D> struct TaCfg {
    static constexpr int kTile = D == 256 ? 64 : 128;             // tokens per step
    static constexpr uint32_t kItemBytes = kTile * D * 2;         // K or V of a step
    static constexpr int kKStages = D == 64 ? 6 : D == 128 ? 3 : 2;
    static constexpr int kVStages = D == 64 ? 6 : 3;
    static constexpr uint32_t kGroupStride = 8 * D * 2;           // 8 token rows, all of head_dim
    static constexpr uint32_t kQBytes = kTaRows * D * 2;          // [D / 64][128 rows][128 B], swizzled
    static constexpr uint32_t kQBlock = kTaRows * 128;
    static constexpr uint32_t kOffK = 0;
    static constexpr uint32_t kOffV = kOffK + kKStages * kItemBytes;
    static constexpr uint32_t kOffQ = kOffV + kVStages * kItemBytes;
    static constexpr uint32_t kOffBar = kOffQ + kQBytes;
    static constexpr uint32_t kOffMax = kOffBar + 1024;           // maxima, [tile parity][half][128 rows]
    static constexpr uint32_t kSmem = kOffMax + 2048;
    static constexpr int kOBufs = D == 256 ? 1 : 2;
    static constexpr uint32_t kColS = kOBufs * D;                 // two S buffers of kTile columns
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kColS + 2 * kTile <= kTmemCols, "TMEM columns");
};

// What the roles need to know of a slice.
struct TaSlice {
    int32_t b, g;          // row, kv head
    int32_t first;         // token of the row's node 0
    int32_t node0, nodes;  // first node of the unit, nodes of the row
    int32_t len;           // cached tokens
    int32_t tok0, tok1;    // the slice's tokens
    int32_t flags;         // kBegins, kEnds, kOver
};
constexpr int kBegins = 1, kEnds = 2, kOver = 4; // it starts / ends the unit; no more slices

struct TaBars {
    uint64_t k_full[6], v_full[6];
    uint64_t p_full[6];       // P of the tile whose V is in slot i written, and that V looked through
    uint64_t s_full[6];       // S of the tile in K slot i is complete: K is free, too
    uint64_t o_done[6];       // P V of the tile in V slot i is complete: V is free, too
    uint64_t q_full;
    uint64_t o_free[2];
    uint64_t o_last[2];       // O of a slice (by its parity) is complete
    uint64_t ml_full[2], ml_free[2]; // (ref, l) of a slice written / read
    uint64_t pair[4];         // the two softmax warps of each TMEM lane quarter
    uint64_t slice_full[kSlices], slice_empty[kSlices];
    uint64_t drain;
    TaSlice slice[kSlices];
    uint8_t bad[kSlices];       // a page of the slice is out of range
    uint8_t nonfinite[kSlices]; // bit w: of drafted tokens 32 w .. 32 w + 31, V of some holds an infinity or NaN
    uint32_t tmem_base;
    int32_t abort;
    int32_t mending; // finishing warps that read a slice's values again
};
static_assert(sizeof(TaBars) <= 1024, "barrier block");

struct TaParams {
    const int32_t *indptr, *mask, *table, *seqlens;
    const __nv_bfloat16 *v_cache;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *err_flag;
    int4 *records;     // [CTA]
    float2 *row_ml;    // [CTA][slice parity][half][128 rows]: from the softmax to the finishing warps
    float2 *part_ml;   // [2 * CTA][slot_rows]
    float *part_o;     // [2 * CTA][slot_rows][D]
    int batch, num_q_heads, num_kv_heads, group, total_q, max_blocks, max_nodes, words;
    int page_shift, box_shift, num_pages, layout;
    int q_tile;        // nodes per unit
    int slot_rows;
    uint32_t q_box_bytes;
    float q_scale;
    int pdl;
    int pair;          // 1: two CTAs side by side on a row's units
    uint32_t k65536;   // 65536: a shift by 16 as a multiplication, in the FMA pipe beside the busy ALU
    bool wide;         // out is 32-byte aligned
};

struct TaMaps {
    CUtensorMap k, v, q;
};

// ---------------------------------------------------------------- work line

struct TaRow {
    int first;  // token of node 0
    int nodes;
    int len;    // cached tokens
    int blocks; // 64-token blocks of keys; 0: the row's output is zeroed
    int tiles;  // units per kv head
    int err;
};

// What a row's part in the call is made from.
struct TaRaw {
    int first, end, len;
};
__device__ __forceinline__ TaRaw ta_raw(const TaParams &p, int b)
{
    b = max(0, min(b, p.batch - 1));
    return {p.indptr[b], p.indptr[b + 1], p.seqlens[b]};
}

// A row's part in the call (see include/pkv.h); tiles = 0 when it owns no node.
__device__ __forceinline__ TaRow ta_row(const TaParams &p, const TaRaw &raw)
{
    TaRow r;
    r.first = raw.first;
    const int64_t n = (int64_t)raw.end - r.first;
    r.len = raw.len;
    r.err = 0;
    r.blocks = 0;
    r.nodes = 0;
    r.tiles = 0;
    if (r.first < 0 || n < 0 || n > (int64_t)p.total_q - r.first) {
        r.err = PKV_ERR_QLEN;
        return r;
    }
    r.nodes = (int)n;
    r.tiles = (r.nodes + p.q_tile - 1) / p.q_tile;
    const int64_t keys = (int64_t)r.len + n;
    if (n > p.max_nodes)
        r.err = PKV_ERR_QLEN;
    else if (r.len >= 0 && keys > min((int64_t)p.max_blocks << p.page_shift, (int64_t)kTreeMaxKeys))
        r.err = PKV_ERR_OVERFLOW;
    else if (r.len >= 0 && n > 0)
        r.blocks = (int)((keys + kTaBlock - 1) / kTaBlock);
    if (n == 0)
        r.err = 0;
    return r;
}

// Block at which a cut `x` positions into a unit of `blocks` blocks falls.
__device__ __forceinline__ int ta_cut(int64_t x, int blocks)
{
    const int64_t k = x - kStartCost;
    if (k < kMinBlocks)
        return 0;
    return blocks - k < kMinBlocks ? blocks : (int)k;
}

// ---------------------------------------------------------------- waits

__device__ __noinline__ bool ta_wait_slow(uint64_t *bar, uint32_t parity, TaBars &bars, int32_t *err_flag)
{
    uint64_t start = globaltimer_ns();
    volatile int32_t *abort = &bars.abort, *mending = &bars.mending;
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity))
                return true;
        if (*abort != 0)
            return false;
        if (*mending != 0) // a bounded loop over a slice, whose length has no bearing on the limit
            start = globaltimer_ns();
        if (globaltimer_ns() - start > kWaitLimitNs) {
            *abort = 1;
            set_error(err_flag, PKV_ERR_TIMEOUT);
            return false;
        }
    }
}

// Bounded wait for the phase of the given parity; gives up when another role has.
__device__ __forceinline__ bool ta_wait(uint64_t *bar, uint32_t parity, TaBars &bars, int32_t *err_flag)
{
    if (mbar_try_wait(bar, parity))
        return true;
    return ta_wait_slow(bar, parity, bars, err_flag);
}
// The same for a whole warp: all lanes get the same answer.
__device__ __forceinline__ bool ta_wait_all(uint64_t *bar, uint32_t parity, TaBars &bars, int32_t *err_flag)
{
    return __all_sync(0xffffffffu, ta_wait(bar, parity, bars, err_flag));
}

// ---------------------------------------------------------------- slices

// Where a CTA's range starts, and its length in positions.
struct TaStart {
    int64_t off, left; // position within the unit, positions of the range
    int b, unit;       // row, unit (with p.pair: two units, one for each CTA) within the row
    TaRow row;
};

// Which of the CTAs of a pair this is, and the index of the pair.
__device__ __forceinline__ int ta_member(const TaParams &p)
{
    return p.pair && blockIdx.x >= gridDim.x >> 1 ? 1 : 0;
}
__device__ __forceinline__ int ta_index(const TaParams &p)
{
    return (int)blockIdx.x - ta_member(p) * (int)(gridDim.x >> 1);
}

// Zeros and -inf for a unit of a row that is inactive or in error.  A whole warp.
template <int D>
__device__ void ta_zero_unit(const TaParams &p, const TaRow &row, int g, int node0, int lane)
{
    const int rows = min(p.q_tile, row.nodes - node0) * p.group;
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        const int64_t at = ((int64_t)row.first + node0 + r / p.group) * p.num_q_heads + g * p.group + r % p.group;
        if (lane < D / 8)
            *reinterpret_cast<uint4 *>(p.out + at * D + lane * 8) = make_uint4(0u, 0u, 0u, 0u);
        if (lane == 0 && p.lse != nullptr)
            p.lse[at] = -INFINITY;
    }
}

// Cuts a CTA's range into slices, in order; units without keys to read are
// finished here.  A whole warp.
template <int D> struct TaWalk {
    TaStart at;
    TaRow row;
    TaRaw then; // the next row, read ahead
    int n; // slices handed out
    bool over;

    __device__ __forceinline__ void start(const TaParams &p, const TaStart &from)
    {
        at = from;
        row = at.row;
        then = ta_raw(p, at.b + 1);
        n = 0;
        over = false;
    }
    // Hands out the next slice (its slot is free).
    __device__ __forceinline__ void publish(const TaParams &p, TaBars &bars, int lane)
    {
        TaSlice s;
        s.flags = kOver;
#pragma unroll 1
        while (at.left > 0) {
            if (at.unit >= row.tiles * p.num_kv_heads >> p.pair) {
                ++at.b;
                at.unit = 0;
                at.off = 0;
                row = ta_row(p, then);
                then = ta_raw(p, at.b + 1);
                continue;
            }
            const int64_t size = kStartCost + row.blocks, take = min(size - at.off, at.left);
            const bool at_start = at.off == 0, at_end = at.off + take >= size;
            const int a = ta_cut(at.off, row.blocks), z = at_end ? row.blocks : ta_cut(at.off + take, row.blocks);
            const int unit = (at.unit << p.pair) + ta_member(p);
            at.left -= take;
            at.off += take;
            if (at_end) {
                ++at.unit;
                at.off = 0;
            }
            if (row.blocks > 0 && a >= z)
                continue;
            // units of a row: row tiles of a kv head next to one another (their K/V stay in L2)
            const int g = unit / row.tiles, node0 = (unit - g * row.tiles) * p.q_tile;
            if (row.blocks == 0) {
                if (at_start) {
                    if (unit == 0 && lane == 0)
                        set_error(p.err_flag, row.err);
                    ta_zero_unit<D>(p, row, g, node0, lane);
                }
                continue;
            }
            s.b = at.b;
            s.g = g;
            s.first = row.first;
            s.node0 = node0;
            s.nodes = row.nodes;
            s.len = row.len;
            s.tok0 = a * kTaBlock;
            s.tok1 = min(z * kTaBlock, row.len + row.nodes);
            s.flags = (a == 0 ? kBegins : 0) | (z == row.blocks ? kEnds : 0);
            break;
        }
        const int slot = n % kSlices;
        if (lane == 0) {
            bars.slice[slot] = s;
            bars.bad[slot] = bars.nonfinite[slot] = 0;
            mbar_arrive(&bars.slice_full[slot]);
        }
        over = (s.flags & kOver) != 0;
        ++n;
    }
};

// The n-th slice; a role that gave up sees the end.
__device__ __forceinline__ TaSlice ta_slice(const TaParams &p, TaBars &bars, int n)
{
    TaSlice s;
    if (ta_wait_all(&bars.slice_full[n % kSlices], (uint32_t)(n / kSlices) & 1, bars, p.err_flag))
        s = bars.slice[n % kSlices];
    else
        s.flags = kOver;
    return s;
}
__device__ __forceinline__ void ta_slice_done(TaBars &bars, int n, int lane)
{
    __syncwarp();
    if (lane == 0)
        mbar_arrive(&bars.slice_empty[n % kSlices]);
}

// The tiles of the slices, one after the other, for a warp that looks at one
// slice at a time.
template <int D> struct TaTiles {
    TaSlice s;
    int n;    // index of the slice
    int tok;  // first token of the tile

    __device__ __forceinline__ void start()
    {
        n = -1;
        tok = s.tok1 = 0;
    }
    __device__ __forceinline__ bool next(const TaParams &p, TaBars &bars, int lane, bool done = true)
    {
        tok += TaCfg<D>::kTile;
        if (tok < s.tok1)
            return true;
        if (n >= 0 && done)
            ta_slice_done(bars, n, lane);
        s = ta_slice(p, bars, ++n);
        tok = s.tok0;
        return !(s.flags & kOver);
    }
    __device__ __forceinline__ bool first() const { return tok == s.tok0; }
};

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// ---------------------------------------------------------------- loads

// One warp loads all K (or all V) tiles of the CTA, one box per lane: boxes of
// min(page, 64) tokens, at most kTile / 8 = 16.  A page id outside the pool
// loads nothing and marks the slice.  The K warp also loads Q: the slot of
// tile T + kKStages - 1 is free when S of tile T - 1 is done, which is when a
// slice that begins with tile T may have the Q buffer.
template <int D, bool IS_K>
__device__ void ta_load(const TaParams &p, const TaMaps &maps, uint8_t *smem, TaBars &bars, int lane)
{
    using C = TaCfg<D>;
    constexpr int kStages = IS_K ? C::kKStages : C::kVStages;
    const CUtensorMap *map = IS_K ? &maps.k : &maps.v;
    uint8_t *ring = smem + (IS_K ? C::kOffK : C::kOffV);
    uint64_t *full = IS_K ? bars.k_full : bars.v_full, *empty = IS_K ? bars.s_full : bars.o_done;
    const int bsh = p.box_shift, boxes = C::kTile >> bsh;
    const uint32_t box_bytes = (uint32_t)(1 << bsh) * D * 2;
    const bool nhd = p.layout == PKV_NHD;
    TaTiles<D> t;
    t.start();
    int q_slice = 0, q_tile0 = 0; // next slice whose Q is due, its first tile
    int slot = 0, issued = 0, issued_slices = 0;
    uint32_t round = 0; // times the ring has been filled
    bool more = true;
    int id = 0; // this lane's page of the coming tile
#pragma unroll 1
    for (int x = 0;; ++x) {
        more = more && t.next(p, bars, lane, !IS_K);
        if (!more && (!IS_K || x >= issued + kStages - 1))
            break;
        if (more && p.pdl && t.tok + C::kTile > t.s.len) // drafted tokens: this call's append has put them there
            asm volatile("griddepcontrol.wait;" ::: "memory");
        const int tok = t.tok + (lane << bsh);
        const bool want = more && lane < boxes && tok < t.s.tok1;
        const int32_t *row = p.table + (int64_t)t.s.b * p.max_blocks;
        if (more && (t.first() || x == 0))
            id = want ? row[tok >> p.page_shift] : 0;
        if (round > 0 && !ta_wait_all(&empty[slot], (round - 1) & 1, bars, p.err_flag))
            break;
        if (more) {
            const bool good = want && id >= 1 && id < p.num_pages;
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, good));
            if (__any_sync(0xffffffffu, want && !good) && IS_K && lane == 0)
                *(volatile uint8_t *)&bars.bad[t.n % kSlices] = 1;
            if (lane == 0)
                mbar_arrive_expect_tx(&full[slot], n * box_bytes);
            __syncwarp();
            if (good) {
                const int in_page = tok & ((1 << p.page_shift) - 1);
                const int c3 = nhd ? ((id << p.page_shift) + in_page) >> 3 : in_page >> 3;
                const int c4 = nhd ? t.s.g : id * p.num_kv_heads + t.s.g;
                tma_load_5d_plain(ring + slot * C::kItemBytes + lane * box_bytes, map, 0, 0, 0, c3, c4, &full[slot]);
            }
            ++issued;
            issued_slices = t.n + 1;
            const int then = tok + C::kTile; // the pages of the slice's next tile, a step ahead
            id = lane < boxes && then < t.s.tok1 ? row[then >> p.page_shift] : 0;
        }
        if (IS_K) {
            if (more && t.first() && x > 0 && lane < D / 64) // a slice's Q into L2 before its buffer is free
                tma_prefetch_3d(&maps.q, lane * 64, t.s.g * p.group, t.s.first + t.s.node0);
            // Q: of the first slice at once, of the others kStages - 1 tiles on
            if (q_slice < issued_slices && (q_slice == 0 || x >= q_tile0 + kStages - 1)) {
                const TaSlice s = bars.slice[q_slice % kSlices];
                if (lane == 0)
                    mbar_arrive_expect_tx(&bars.q_full, p.q_box_bytes * (D / 64));
                __syncwarp();
                if (lane < D / 64)
                    tma_load_3d_plain(smem + C::kOffQ + lane * C::kQBlock, &maps.q, lane * 64, s.g * p.group,
                                      s.first + s.node0, &bars.q_full);
                q_tile0 += (s.tok1 - s.tok0 + C::kTile - 1) / C::kTile;
                ta_slice_done(bars, q_slice, lane);
                ++q_slice;
            }
        }
        if (++slot == kStages) {
            slot = 0;
            ++round;
        }
    }
    // Copies still in flight (a role gave up): they land before the CTA ends.
#pragma unroll 1
    for (int k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
        mbar_wait(&full[k % kStages], (uint32_t)(k / kStages) & 1);
    if (q_slice > 0)
        mbar_wait(&bars.q_full, (uint32_t)(q_slice - 1) & 1);
}

__device__ __forceinline__ bool bf16_nonfinite(uint32_t half)
{
    return (half & 0x7f80u) == 0x7f80u;
}

// The i-th 16-byte piece of a V tile in shared memory, row by row (D / 8 pieces
// a row; which piece of the row it is, the swizzle decides).
template <int D> __device__ __forceinline__ uint8_t *ta_v_piece(uint8_t *vb, int i)
{
    const int row = i / (D / 8), piece = i % (D / 8);
    return vb + (row >> 3) * TaCfg<D>::kGroupStride + (piece >> 3) * 1024 + (row & 7) * 128 + (piece & 7) * 16;
}

// One warp hands out the slices, as far ahead as there is room, and looks V
// through before the MMAs read it.  Of a tile with drafted tokens it replaces
// their infinities and NaN by 0 (and marks the slice); rows past the keys, up
// to the multiple of 16 that the MMAs read, become 0.
template <int D>
__device__ void ta_walk(const TaParams &p, uint8_t *smem, TaBars &bars, const TaStart &from, int lane)
{
    using C = TaCfg<D>;
    constexpr int kPieces = D / 8; // 16-byte pieces of a row
    TaWalk<D> walk;
    walk.start(p, from);
    int n = 0, v_slot = 0; // the slice at hand
    uint32_t v_par = 0;
    TaSlice s;
    s.tok1 = s.len = 0;
    int tok = 0;
#pragma unroll 1
    for (;;) {
#pragma unroll 1
        while (!walk.over) {
            uint64_t *empty = &bars.slice_empty[walk.n % kSlices];
            const uint32_t parity = (uint32_t)(walk.n / kSlices - 1) & 1;
            if (walk.n >= kSlices && !__all_sync(0xffffffffu, mbar_test_wait(empty, parity))) {
                if (walk.n > n)
                    break;
                if (!ta_wait_all(empty, parity, bars, p.err_flag))
                    return;
            }
            walk.publish(p, bars, lane);
        }
        if (tok >= s.tok1) {
            s = ta_slice(p, bars, n);
            if (s.flags & kOver)
                return;
            tok = s.tok0;
        }
        if (!ta_wait_all(&bars.v_full[v_slot], v_par, bars, p.err_flag))
            return;
        const int tokens = min(C::kTile, s.tok1 - tok);
        const int d0 = min(tokens, max(0, s.len - tok)), r1 = (tokens + 15) & ~15;
        if (d0 < r1) {
            uint8_t *vb = smem + C::kOffV + v_slot * C::kItemBytes;
            // any infinity or NaN: 0 * x is NaN, and stays in the sum
            __nv_bfloat162 sum = __floats2bfloat162_rn(0.f, 0.f);
            const __nv_bfloat162 zero = sum;
#pragma unroll 4
            for (int i = d0 * kPieces + lane; i < tokens * kPieces; i += 32) {
                const uint4 x = *reinterpret_cast<const uint4 *>(ta_v_piece<D>(vb, i));
                sum = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.x), zero, sum);
                sum = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.y), zero, sum);
                sum = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.z), zero, sum);
                sum = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.w), zero, sum);
            }
            if (__any_sync(0xffffffffu, __hisnan(sum.x) || __hisnan(sum.y))) {
                uint32_t words = 0;
#pragma unroll 1
                for (int i = d0 * kPieces + lane; i < tokens * kPieces; i += 32) {
                    uint32_t *w = reinterpret_cast<uint32_t *>(ta_v_piece<D>(vb, i));
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t keep = (bf16_nonfinite(w[k]) ? 0xffff0000u : 0xffffffffu) &
                                              (bf16_nonfinite(w[k] >> 16) ? 0xffffu : 0xffffffffu);
                        w[k] &= keep;
                        words |= keep != 0xffffffffu ? 1u << ((tok + i / kPieces - s.len) >> 5) : 0u;
                    }
                }
                words = __reduce_or_sync(0xffffffffu, words);
                if (lane == 0) {
                    volatile uint8_t *set = &bars.nonfinite[n % kSlices];
                    *set = (uint8_t)(*set | words);
                }
            }
            for (int i = tokens * kPieces + lane; i < r1 * kPieces; i += 32)
                *reinterpret_cast<uint4 *>(ta_v_piece<D>(vb, i)) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem(); // before the MMAs' reads
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bars.p_full[v_slot]);
        if (++v_slot == C::kVStages) {
            v_slot = 0;
            v_par ^= 1;
        }
        tok += C::kTile;
        if (tok >= s.tok1)
            ta_slice_done(bars, n++, lane);
    }
}

// ---------------------------------------------------------------- MMA

// The MMA warp runs as a whole, so that descriptors stay in uniform registers;
// one elected thread (always the same) issues.
// Four MMAs of 64 values of the inner dimension: A and B 32 bytes on each time.
__device__ __forceinline__ void ta_mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
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
// The MMAs of 16 keys: P's hi parts, then the lo parts 16 columns on.
__device__ __forceinline__ void ta_mma_pv(uint32_t o, uint32_t a, uint64_t v, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred e, p, t;\n\t"
                 ".reg .b32 a1;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.eq.b32 t, 0, 0;\n\t"
                 "add.u32 a1, %1, 16;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], %2, %3, t;\n\t}" ::"r"(o),
                 "r"(a), "l"(v), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// The MMAs of 32 keys; V is 16 keys on after the first two.
template <uint32_t STEP>
__device__ __forceinline__ void ta_mma_pv2(uint32_t o, uint32_t a, uint64_t v, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred e, p, t;\n\t"
                 ".reg .b32 a1, a2, a3;\n\t"
                 ".reg .b64 v1;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.eq.b32 t, 0, 0;\n\t"
                 "add.u32 a1, %1, 16;\n\tadd.u32 a2, %1, 8;\n\tadd.u32 a3, %1, 24;\n\t"
                 "add.s64 v1, %2, %5;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], %2, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], v1, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], v1, %3, t;\n\t}" ::"r"(o),
                 "r"(a), "l"(v), "r"(idesc), "r"(accumulate), "n"(STEP)
                 : "memory");
}
__device__ __forceinline__ void ta_commit(uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred e;\n\t"
                 "elect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                     smem_addr(bar))
                 : "memory");
}

template <int D>
__device__ void ta_mma(const TaParams &p, uint8_t *smem, TaBars &bars, uint32_t tmem, int lane)
{
    using C = TaCfg<D>;
    constexpr uint32_t kIdescS = tc_idesc_bf16(kTaRows, C::kTile, false, false);
    constexpr uint32_t kIdescO = tc_idesc_bf16(kTaRows, D, false, true);
    const uint64_t kd0 = tc_sw128_desc(smem_addr(smem + C::kOffK), 16, C::kGroupStride);
    const uint64_t vd0 = tc_sw128_desc(smem_addr(smem + C::kOffV), 1024, C::kGroupStride);
    const uint64_t qd0 = tc_sw128_desc(smem_addr(smem + C::kOffQ), 16, 1024);
    // The walk over tiles in warp-uniform registers (a value that one lane read is
    // uniform to the compiler): TMEM addresses and descriptors then need no move
    // into uniform registers at every MMA.
    int n = 0, tok = 0, tok0 = 0, tok1 = 0, gt = 0;
    auto open = [&] { // slice n
        const TaSlice s = ta_slice(p, bars, n);
        tok = tok0 = __shfl_sync(0xffffffffu, s.tok0, 0);
        tok1 = __shfl_sync(0xffffffffu, s.tok1, 0);
        return !__shfl_sync(0xffffffffu, s.flags & kOver, 0);
    };
    bool issued = false, more = open();
    int prev = -1; // tile whose P V is due
    int prev_tokens = 0, prev_unit = 0;
    bool prev_first = false, prev_last = false;
    int k_slot = 0, v_slot = 0;
    uint32_t k_par = 0, v_par = 0;
#pragma unroll 1
    while (more || prev >= 0) {
        if (more) { // S of the next tile
            if (((tok == tok0) && !ta_wait_all(&bars.q_full, (uint32_t)n & 1, bars, p.err_flag)) ||
                !ta_wait_all(&bars.k_full[k_slot], k_par, bars, p.err_flag))
                break;
            tc_fence_after();
            issued = true;
            const uint32_t d = tmem + C::kColS + (uint32_t)(gt & 1) * C::kTile;
            const uint64_t kd = kd0 + (uint64_t)(k_slot * C::kItemBytes >> 4);
#pragma unroll 1
            for (int blk = 0; blk < D / 64; ++blk)
                ta_mma_ss4(d, qd0 + (uint64_t)(blk * C::kQBlock >> 4), kd + (uint64_t)(blk * 1024 >> 4), kIdescS,
                           blk > 0 ? 1u : 0u);
            ta_commit(&bars.s_full[k_slot]);
            if (++k_slot == C::kKStages) {
                k_slot = 0;
                k_par ^= 1;
            }
        }
        if (prev >= 0) { // O += P V of the one before
            const uint32_t ob = C::kOBufs == 1 ? 0 : prev_unit & 1;
            const uint32_t use = C::kOBufs == 1 ? prev_unit : prev_unit >> 1;
            if ((prev_first && use > 0 && !ta_wait_all(&bars.o_free[ob], (use - 1) & 1, bars, p.err_flag)) ||
                !ta_wait_all(&bars.p_full[v_slot], v_par, bars, p.err_flag))
                break;
            tc_fence_after();
            const uint32_t o = tmem + ob * D;
            uint32_t a = tmem + C::kColS + (uint32_t)(prev & 1) * C::kTile;
            uint64_t vd = vd0 + (uint64_t)(v_slot * C::kItemBytes >> 4);
            int k = 0;
            constexpr uint32_t kStep = 2 * C::kGroupStride >> 4; // 16 keys of V
#pragma unroll 1
            for (; k + 16 < prev_tokens; k += 32) {
                ta_mma_pv2<kStep>(o, a, vd, kIdescO, !prev_first || k > 0 ? 1u : 0u);
                vd += 2 * kStep;
                a += 32;
            }
            if (k < prev_tokens)
                ta_mma_pv(o, a, vd, kIdescO, !prev_first || k > 0 ? 1u : 0u);
            ta_commit(&bars.o_done[v_slot]);
            if (prev_last)
                ta_commit(&bars.o_last[prev_unit & 1]);
            if (++v_slot == C::kVStages) {
                v_slot = 0;
                v_par ^= 1;
            }
        }
        prev = -1;
        if (more) {
            prev = gt;
            prev_tokens = min(C::kTile, tok1 - tok);
            prev_first = (tok == tok0);
            prev_last = tok + C::kTile >= tok1;
            prev_unit = n;
            ++gt;
            tok += C::kTile;
            if (tok >= tok1) {
                ta_slice_done(bars, n++, lane);
                more = open();
            }
        }
    }
    if (issued) {
        ta_commit(&bars.drain);
        mbar_wait(&bars.drain, 0);
    }
}

// ---------------------------------------------------------------- softmax

__device__ __forceinline__ void tmem_st16_issue(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
// Three-input maximum (one instruction).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Which of the drafted keys 32 w .. 32 w + 31 a node sees (w < 0: cached
// keys, all of them; none at and past `nodes`).
__device__ __forceinline__ uint32_t ta_mask_word(const int32_t *mask, int nodes, int w)
{
    if (w < 0)
        return 0xffffffffu;
    const int rest = nodes - w * 32;
    if (rest <= 0)
        return 0u;
    const uint32_t x = (uint32_t)mask[w];
    return rest >= 32 ? x : x & ((1u << rest) - 1u);
}

// 32 bytes to global memory; one store where the address allows it (`wide`).
__device__ __forceinline__ void store32(void *dst, const uint32_t *w, bool wide)
{
    if (!wide) {
        static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Columns col .. col + 7 of V of a token in the cache; zeros for a page that is none.
template <int D>
__device__ __forceinline__ uint4 ta_cached_v(const TaParams &p, int b, int g, int tok, int col)
{
    const int64_t page = p.table[(int64_t)b * p.max_blocks + (tok >> p.page_shift)];
    if (page < 1 || page >= p.num_pages)
        return make_uint4(0u, 0u, 0u, 0u);
    const int64_t slot = tok & ((1 << p.page_shift) - 1);
    const int64_t at = p.layout == PKV_NHD ? (((page << p.page_shift) + slot) * p.num_kv_heads + g) * D
                                           : (((page * p.num_kv_heads + g) << p.page_shift) + slot) * D;
    return *reinterpret_cast<const uint4 *>(p.v_cache + at + col);
}

// Adds to a node's O the infinities and NaN that the drafted tokens j0 .. j1 - 1
// it sees hold (rare; read again from the cache).  `words`: which 32 tokens to
// look at; of them only those that some lane sees are read, so that padding
// costs a vote.  A whole warp; lanes with `live` false change nothing.  Whether
// any O changed.
template <int D>
__device__ __noinline__ bool ta_add_nonfinite(const TaParams &p, int b, int len, int g, const int32_t *mask, int j0, int j1,
                                              uint32_t words, bool live, uint32_t o_col, int lane)
{
    bool changed = false;
#pragma unroll 1
    for (; words != 0; words &= words - 1) {
        const int first = (__ffs(words) - 1) * 32, lo = max(j0 - first, 0), hi = min(j1 - first, 32);
        if (lo >= hi)
            continue;
        const uint32_t mine = live ? (uint32_t)mask[first >> 5] & (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo) : 0u;
#pragma unroll 1
        for (uint32_t keys = __reduce_or_sync(0xffffffffu, mine); keys != 0; keys &= keys - 1) {
            const int k = __ffs(keys) - 1;
            const uint4 x = ta_cached_v<D>(p, b, g, len + first + k, lane % (D / 8) * 8);
            uint32_t w[4] = {x.x, x.y, x.z, x.w}, any = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] &= (bf16_nonfinite(w[e]) ? 0xffffu : 0u) | (bf16_nonfinite(w[e] >> 16) ? 0xffff0000u : 0u);
                any |= w[e];
            }
            const uint32_t pieces = __ballot_sync(0xffffffffu, any != 0);
            if (pieces == 0)
                continue;
            changed = true;
            const bool sees = mine >> k & 1u;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                if (!(pieces >> (c >> 3) & 0xfu))
                    continue;
                uint32_t o[32];
                tmem_ld32(o_col + c, o);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const uint32_t v = __shfl_sync(0xffffffffu, w[(i & 7) >> 1], (c + i) >> 3);
                    if (sees) {
                        o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(v << 16));
                        o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) + __uint_as_float(v & 0xffff0000u));
                    }
                }
                __syncwarp();
                tmem_st32(o_col + c, o);
            }
        }
    }
    return changed;
}

// O of a slice with infinities or NaN among its cached values.  A weight goes
// into the MMAs as two parts whose second may be negative or 0, so such a value
// arrives as a NaN or an infinity of either sign; all that is certain is that
// it is not finite.  The columns where it is not become the sum of the slice's
// cached values there that are not finite, which is what the formula gives for
// positive weights, the same for every node.  A whole warp, rare: it reads such
// columns of the slice's V again, 8 at a time, a token per lane.  64 uneven rows
// with an infinity in one column of the longest take 0.41 ms a call for 0.15
// (2.2 with all columns read), with a token that is NaN throughout 0.58 (2.6
// without the look at columns that are NaN already).  Lanes with `mend` false
// change nothing.
constexpr int kMendTokens = 2048; // between looks at whether all 8 columns are NaN
template <int D>
__device__ __noinline__ void ta_mend_cached(const TaParams &p, int b, int g, int tok0, int tok1, bool mend, uint32_t o_col,
                                            int lane)
{
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t odd = 0;
        {
            uint32_t o[32];
            tmem_ld32(o_col + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                odd |= mend && (o[i] & 0x7f800000u) == 0x7f800000u ? 1u << i : 0u;
        }
        odd = __reduce_or_sync(0xffffffffu, odd);
#pragma unroll 1
        while (odd != 0) {
            const int in = (__ffs(odd) - 1) & ~7, col = c + in;
            odd &= ~(0xffu << in);
            float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            uint32_t nan = 0; // columns that are NaN already
#pragma unroll 1
            for (int64_t t0 = tok0; t0 < tok1 && nan != 0xffu; t0 += kMendTokens) {
                const int end = (int)min(t0 + kMendTokens, (int64_t)tok1);
#pragma unroll 4
                for (int tok = (int)t0 + lane; tok < end; tok += 32) {
                    const uint4 x = ta_cached_v<D>(p, b, g, tok, col);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum[2 * e] += bf16_nonfinite(w[e]) ? __uint_as_float(w[e] << 16) : 0.f;
                        sum[2 * e + 1] += bf16_nonfinite(w[e] >> 16) ? __uint_as_float(w[e] & 0xffff0000u) : 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    nan |= isnan(sum[e]) ? 1u << e : 0u;
                nan = __reduce_or_sync(0xffffffffu, nan);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
                uint32_t x;
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                             : "=r"(x)
                             : "r"(o_col + col + e)
                             : "memory");
                x = mend && sum[e] != 0.f && (x & 0x7f800000u) == 0x7f800000u ? __float_as_uint(sum[e]) : x;
                asm volatile(
                    "tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(
                        o_col + col + e),
                    "r"(x)
                    : "memory");
            }
        }
    }
}

// The softmax: two threads per MMA row, each on half of a tile's columns and
// (where O is rescaled) half of O's.
template <int D>
__device__ void ta_softmax(const TaParams &p, uint8_t *smem, TaBars &bars, uint32_t tmem, int warp, int lane)
{
    using C = TaCfg<D>;
    constexpr int kChunks = C::kTile / 64;      // 32-column chunks of this thread
    const int half = (warp - kTaSoftmaxWarp) >> 2;
    const int quarter = warp & 3; // TMEM lanes this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
    float *maxima = reinterpret_cast<float *>(smem + C::kOffMax);
    const float qs = p.q_scale, qse = qs > 0.f ? qs : 1.f;
    const int node_in_tile = r / p.group;
    int gt = 0;          // tiles before this one
    int k_slot = 0, v_slot = 0;
    uint32_t k_par = 0;
    uint32_t meetings = 0; // of the two warps of this quarter

#pragma unroll 1
    for (int n = 0;; ++n) {
        const TaSlice s = ta_slice(p, bars, n);
        if (s.flags & kOver)
            return;
        const int rows = min(p.q_tile, s.nodes - s.node0) * p.group; // MMA rows in use
        const bool live = r < rows, warp_live = quarter * 32 < rows;
        const int32_t *mask = p.mask + ((int64_t)s.first + (live ? s.node0 + node_in_tile : 0)) * p.words;
        const uint32_t o_col = t_row + (C::kOBufs == 1 ? 0u : (n & 1) * D);
        const float slack = (float)(33 - __clz(s.len + s.nodes - 1));
        float ref = -INFINITY, l = 0.f; // the weights' reference; this half's part of their sum
#pragma unroll 1
        for (int tok = s.tok0; tok < s.tok1; tok += C::kTile, ++gt) {
            const int tok_h = tok + half * (C::kTile / 2), tokens = s.tok1 - tok_h; // this half's keys
            // tiles with drafted keys or past the slice's end: the node's mask words
            const bool masked = tok + C::kTile > s.len || tok + C::kTile > s.tok1;
            uint32_t words[kChunks + 1];
            if (masked && warp_live) {
                const int w0 = (tok_h - s.len) >> 5;
#pragma unroll
                for (int c = 0; c <= kChunks; ++c)
                    words[c] = ta_mask_word(mask, s.nodes, w0 + c);
            }
            if (!ta_wait_all(&bars.s_full[k_slot], k_par, bars, p.err_flag))
                return;
            if (++k_slot == C::kKStages) {
                k_slot = 0;
                k_par ^= 1;
            }
            tc_fence_after();
            const uint32_t s_col = t_row + C::kColS + (uint32_t)(gt & 1) * C::kTile + half * (C::kTile / 2);
            float alpha = 1.f;
            bool rescale = false;
            if (warp_live) {
                // Tiles with drafted keys or past the slice's end, and scales that
                // cannot be folded into the exponent: S is rewritten once, so that
                // the passes below are the same short loops for every tile.
                if (masked || !(qs > 0.f)) {
                    const float by = qs > 0.f ? 1.f : qs;
                    const int shift = (tok_h - s.len) & 31;
#pragma unroll 1
                    for (int c = 0; c < kChunks; ++c) {
                        const int end = tokens - 32 * c;
                        uint32_t seen = end >= 32 ? 0xffffffffu : end <= 0 ? 0u : (1u << end) - 1u;
                        if (masked) {
                            seen &= __funnelshift_r(words[0], words[1], shift);
#pragma unroll
                            for (int w = 0; w < kChunks; ++w)
                                words[w] = words[w + 1];
                        }
                        uint32_t x[32];
                        tmem_ld32(s_col + 32 * c, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = seen >> i & 1u ? __float_as_uint(__uint_as_float(x[i]) * by) : 0xff800000u;
                        tmem_st32(s_col + 32 * c, x);
                    }
                }
                float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    uint32_t x[32];
                    tmem_ld32(s_col + 32 * c, x);
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        m2[i >> 1 & 1] = max3(m2[i >> 1 & 1], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                }
                float mx = live ? fmaxf(m2[0], m2[1]) * qse : -INFINITY;
                // the row's maximum over both halves
                float *at = maxima + (meetings & 1) * (2 * kTaRows) + r;
                at[half * kTaRows] = mx;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars.pair[quarter]);
                if (!ta_wait_all(&bars.pair[quarter], meetings & 1, bars, p.err_flag))
                    return;
                ++meetings;
                mx = fmaxf(mx, at[(1 - half) * kTaRows]);
                if (mx + slack > ref) {
                    const float next = mx + (slack + kRescaleLog2);
                    rescale = ref != -INFINITY; // before the slice's first P V there is no O
                    alpha = ex2_approx(ref - next);
                    ref = next;
                }
                __syncwarp(); // the loads below are the whole warp's
                float2 sum2 = make_float2(0.f, 0.f);
                const float m_ref = ref == -INFINITY ? 0.f : ref;
                const float2 q2 = make_float2(qse, qse), nm2 = make_float2(-m_ref, -m_ref);
#pragma unroll 1
                for (int c = 0; c < kChunks; ++c) {
                    uint32_t y[32];
                    tmem_ld32(s_col + 32 * c, y);
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 a = ffma2(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), q2,
                                               nm2);
                        const float2 w = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                        sum2 = __fadd2_rn(sum2, w);
                        const __nv_bfloat162 h = __floats2bfloat162_rn(w.x, w.y);
                        const uint32_t hw = *reinterpret_cast<const uint32_t *>(&h);
                        uint32_t h0;
                        asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(h0) : "r"(hw), "r"(p.k65536), "r"(0));
                        const float2 d = ffma2(make_float2(__uint_as_float(h0), __uint_as_float(hw & 0xffff0000u)),
                                               make_float2(-1.f, -1.f), w); // exact
                        const __nv_bfloat162 lw = __floats2bfloat162_rn(d.x, d.y);
                        hi[e] = *reinterpret_cast<const uint32_t *>(&h);
                        lo[e] = *reinterpret_cast<const uint32_t *>(&lw);
                    }
                    tmem_st16_issue(s_col + 32 * c, hi);
                    tmem_st16_issue(s_col + 32 * c + 16, lo);
                }
                tmem_st_wait();
                l = l * alpha + (sum2.x + sum2.y);
            }
            if (__any_sync(0xffffffffu, rescale)) {
                if (!ta_wait_all(&bars.o_done[(gt - 1) % C::kVStages], (uint32_t)((gt - 1) / C::kVStages) & 1, bars,
                                 p.err_flag))
                    return;
                tc_fence_after();
                const float a = rescale ? alpha : 1.f;
#pragma unroll 1
                for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_col + c, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                    tmem_st32(o_col + c, o);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars.p_full[v_slot]);
            if (++v_slot == C::kVStages)
                v_slot = 0;
        }
        // (ref, l) to the warps that finish the slice
        if (n >= 2 && !ta_wait_all(&bars.ml_free[n & 1], (uint32_t)(n / 2 - 1) & 1, bars, p.err_flag))
            return;
        p.row_ml[((int64_t)blockIdx.x * 4 + (n & 1) * 2 + half) * kTaRows + r] = make_float2(ref, l);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bars.ml_full[n & 1]);
        ta_slice_done(bars, n, lane);
    }
}

// A value another warp of this CTA has written (never from an earlier load).
__device__ __forceinline__ float2 load_fresh(const float2 *at)
{
    float2 v;
    asm volatile("ld.volatile.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(at) : "memory");
    return v;
}

// Finishes the slices, one thread per MMA row: O / l to out where the slice is a
// whole unit, else O and (ref, l) to the workspace.
template <int D>
__device__ void ta_finish(const TaParams &p, TaBars &bars, uint32_t tmem, int warp, int lane)
{
    using C = TaCfg<D>;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
    const int node_in_tile = r / p.group, head_in_group = r - node_in_tile * p.group;
    int record = 0;
    int4 tail = make_int4(0, 0, 0, 0);
#pragma unroll 1
    for (int n = 0;; ++n) {
        const TaSlice s = ta_slice(p, bars, n);
        if (s.flags & kOver)
            break;
        const int rows = min(p.q_tile, s.nodes - s.node0) * p.group;
        const bool live = r < rows, warp_live = quarter * 32 < rows;
        const int64_t token = (int64_t)s.first + (live ? s.node0 + node_in_tile : 0);
        const int64_t out_row = token * p.num_q_heads + s.g * p.group + head_in_group;
        const uint32_t parity = (uint32_t)(n >> 1) & 1;
        if (!ta_wait_all(&bars.ml_full[n & 1], parity, bars, p.err_flag))
            return;
        const float2 *ml = p.row_ml + ((int64_t)blockIdx.x * 4 + (n & 1) * 2) * kTaRows + r;
        const float2 a = load_fresh(ml), b = load_fresh(ml + kTaRows);
        const float m = a.x, l = a.y + b.y;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bars.ml_free[n & 1]);
        if (!ta_wait_all(&bars.o_last[n & 1], parity, bars, p.err_flag))
            return;
        tc_fence_after();
        const bool bad = *(volatile uint8_t *)&bars.bad[n % kSlices] != 0;
        const uint32_t nonfinite = *(volatile uint8_t *)&bars.nonfinite[n % kSlices];
        const uint32_t o_col = t_row + (C::kOBufs == 1 ? 0u : (n & 1) * D);
        const bool begins = s.flags & kBegins, ends = s.flags & kEnds, whole = begins && ends;
        const int64_t part = (int64_t)(2 * blockIdx.x + (begins ? 1 : 0)) * p.slot_rows + r;
        const bool zero = bad || l == 0.f;
        const float inv = 1.f / l;
#pragma unroll 1
        for (bool again = false;; again = true) { // twice where V is not finite
            float2 odd = make_float2(0.f, 0.f); // NaN once O is not finite
#pragma unroll 1
            for (int c = 0; warp_live && c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(o_col + c, o);
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        odd = ffma2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])),
                                    make_float2(0.f, 0.f), odd);
                    if (whole) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv,
                                                                           __uint_as_float(o[2 * e + 1]) * inv);
                            w[e] = zero ? 0u : *reinterpret_cast<const uint32_t *>(&h);
                        }
                        store32(p.out + out_row * D + c, w, p.wide);
                        store32(p.out + out_row * D + c + 16, w + 8, p.wide);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            store32(p.part_o + part * D + c + e, o + e, true);
                    }
                }
                __syncwarp(); // the next load is the whole warp's
            }
            if (again || !warp_live)
                break;
            // cached values first, while O shows where they are; not where the scores are NaN
            const bool mend = live && !zero && l < INFINITY && !(odd.x + odd.y == 0.f);
            bool changed = __any_sync(0xffffffffu, mend);
            if (changed) {
                if (lane == 0)
                    atomicAdd(&bars.mending, 1);
                ta_mend_cached<D>(p, s.b, s.g, s.tok0, min(s.tok1, s.len), mend, o_col, lane);
                if (lane == 0)
                    atomicSub(&bars.mending, 1);
            }
            if (nonfinite != 0) {
                if (p.pdl) // V is read from the cache again, where this call's append puts it
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                changed |= ta_add_nonfinite<D>(p, s.b, s.len, s.g, p.mask + token * p.words, max(0, s.tok0 - s.len),
                                               min(s.nodes, s.tok1 - s.len), nonfinite, live, o_col, lane);
            }
            if (!changed)
                break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bars.o_free[C::kOBufs == 1 ? 0 : n & 1]);
        if (live) {
            if (!whole)
                p.part_ml[part] = make_float2(m, l);
            else if (p.lse != nullptr)
                p.lse[out_row] = zero ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        if (r == 0) {
            if (bad)
                set_error(p.err_flag, PKV_ERR_PAGE);
            if (!begins)
                record |= kHeadValid | (ends ? kHeadEnd : 0) | (bad ? kHeadBad : 0);
            else if (!ends) {
                record |= kTail | (bad ? kTailBad : 0);
                tail = make_int4(0, s.first + s.node0, s.g, rows);
            }
        }
        ta_slice_done(bars, n, lane);
    }
    if (r == 0) {
        tail.x = record;
        p.records[blockIdx.x] = tail;
    }
}

// ---------------------------------------------------------------- kernel

// Positions of row b on the work line.
__device__ __forceinline__ int64_t ta_positions(const TaParams &p, const TaRow &r)
{
    return (int64_t)(r.tiles * p.num_kv_heads >> p.pair) * (kStartCost + r.blocks);
}

// a / b for a >= 0, b > 0: 64-bit division only where it is needed (it is long,
// and this is the start of every CTA).
__device__ __forceinline__ int64_t ta_div(int64_t a, int64_t b)
{
    return a >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// This CTA's range, an equal part of all rows' positions: prefix sum over the
// rows (a few consecutive ones per thread), and the thread whose rows the range
// starts in says where.  `scratch`: kTaThreads / 32 sums, then a TaStart.
__device__ TaStart ta_start(const TaParams &p, int64_t *scratch)
{
    constexpr int kPer = (kMaxTreeBatch + kTaThreads - 1) / kTaThreads;
    TaStart *found = reinterpret_cast<TaStart *>(scratch + kTaThreads / 32);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    TaRow row[kPer];
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int b = tid * kPer + i;
        row[i].tiles = row[i].blocks = 0;
        if (b < p.batch) {
            row[i] = ta_row(p, ta_raw(p, b));
            if (blockIdx.x == 0 && row[i].tiles == 0)
                set_error(p.err_flag, row[i].err); // no unit reports it
        }
        sum += ta_positions(p, row[i]);
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
        found->off = found->left = 0;
        found->b = found->unit = 0;
        found->row = row[0];
    }
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kTaThreads / 32; ++w) {
        const int64_t v = scratch[w];
        x += w < warp ? v : 0;
        total += v;
    }
    x -= sum;
    const int most = (int)gridDim.x >> p.pair, c = ta_index(p);
    const int64_t ctas = total >= (int64_t)most * kMinRange ? most : max(1, (int)total / kMinRange);
    if (c < ctas) {
        // as the quotient and remainder of total / ctas, with small numbers
        const int64_t q = ta_div(total, ctas);
        const int rest = (int)(total - q * ctas); // (below 160: products with c stay small)
        const int64_t lo = q * c + rest * c / (int)ctas, hi = q * (c + 1) + rest * (c + 1) / (int)ctas;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t positions = ta_positions(p, row[i]), in_row = lo - x;
            if (hi > lo && in_row >= 0 && in_row < positions) {
                const int size = kStartCost + row[i].blocks;
                TaStart at;
                at.b = tid * kPer + i;
                at.unit = (int)ta_div(in_row, size);
                at.off = in_row - (int64_t)at.unit * size;
                at.left = hi - lo;
                at.row = row[i];
                *found = at;
            }
            x += positions;
        }
    }
    __syncthreads();
    return *found;
}

template <int D>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_attn_kernel(const __grid_constant__ TaParams p, const __grid_constant__ TaMaps maps)
{
    using C = TaCfg<D>;
    extern __shared__ __align__(1024) unsigned char ta_smem_raw[];
    uint8_t *smem = ta_smem_raw;
    if ((smem_addr(smem) & 1023u) != 0) { // the swizzled tiles need it; dynamic shared memory starts so
        set_error(p.err_flag, PKV_ERR_TIMEOUT);
        return;
    }
    TaBars &bars = *reinterpret_cast<TaBars *>(smem + C::kOffBar);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); // the combine kernel waits for this grid
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kKStages; ++i) {
            mbar_init(&bars.k_full[i], 1);
            mbar_init(&bars.s_full[i], 1);
        }
        for (int i = 0; i < C::kVStages; ++i) {
            mbar_init(&bars.v_full[i], 1);
            mbar_init(&bars.p_full[i], 9); // the softmax warps and the one that looks V through
            mbar_init(&bars.o_done[i], 1);
        }
        mbar_init(&bars.q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.o_last[i], 1);
            mbar_init(&bars.o_free[i], 4); // the finishing warps
            mbar_init(&bars.ml_full[i], 8);
            mbar_init(&bars.ml_free[i], 4);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(&bars.pair[i], 2);
        for (int i = 0; i < kSlices; ++i) {
            mbar_init(&bars.slice_full[i], 1);
            mbar_init(&bars.slice_empty[i], kReaders);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = bars.mending = 0;
        mbar_init_fence();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
        prefetch_tensormap(&maps.q);
    }
    if (warp == kTaMmaWarp) {
        tmem_alloc(&bars.tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    // With an append before it this kernel starts beside that: everything earlier
    // is complete, and only K/V at and past a row's length wait for it.
    const TaStart from = ta_start(p, reinterpret_cast<int64_t *>(smem + C::kOffK));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    fence_proxy_async_smem(); // the scratch's reads and writes before the copies over it
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem_base, 0);
    if (threadIdx.x == kTaEndWarp * 32) // the thread that writes it at the end
        p.records[blockIdx.x] = make_int4(0, 0, 0, 0);

    if (warp == kTaWalkWarp)
        ta_walk<D>(p, smem, bars, from, lane);
    else if (warp == kTaKWarp)
        ta_load<D, true>(p, maps, smem, bars, lane);
    else if (warp == kTaVWarp)
        ta_load<D, false>(p, maps, smem, bars, lane);
    else if (warp == kTaMmaWarp)
        ta_mma<D>(p, smem, bars, tmem, lane);
    else if (warp < kTaEndWarp)
        ta_softmax<D>(p, smem, bars, tmem, warp, lane);
    else
        ta_finish<D>(p, bars, tmem, warp, lane);

    if (p.pdl && warp == kTaKWarp) // this grid ends after the append, whether it read its tokens or not
        asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kTaMmaWarp)
        tmem_dealloc(tmem, C::kTmemCols);
}

// ---------------------------------------------------------------- combine

constexpr int kCombineThreads = 256;

// x * w; an infinity stays one where its weight is nothing in 32 bits.
__device__ __forceinline__ float ta_weighed(float x, float w)
{
    return fabsf(x) == INFINITY ? x : x * w;
}

// Joins the slices of the unit that CTA blockIdx.x began and did not end: out =
// sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s (m_s the slice's ref), over the
// CTAs after it up to the one that ended it, in that order.  D / 8 threads per
// MMA row; gridDim.y blocks take one row per thread, so that all of a thread's
// loads are under way at once: what bounds this kernel is the chain record,
// (ref, l) and O (4.5 us for 32 rows of 512 .. 1024 tokens with trees of 16
// nodes).
template <int D>
__global__ void __launch_bounds__(kCombineThreads) tree_combine_kernel(const __grid_constant__ TaParams p, int ctas)
{
    const int c0 = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    constexpr int kPerRow = D / 8;
    const int col = tid % kPerRow * 8, row = blockIdx.y * (kCombineThreads / kPerRow) + tid / kPerRow;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 rec = p.records[c0];
    int flags = c0 + 1 + lane < ctas ? p.records[c0 + 1 + lane].x : 0; // of the 32 CTAs after it
    if (!(rec.x & kTail))
        return;
    const int64_t at_row = min(row, rec.w - 1); // (whole warps go on: they vote)
    float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    int bad = rec.x & kTailBad;
    constexpr int kAtOnce = 4;
    int slot[kAtOnce] = {2 * c0 + 1, -1, -1, -1}, n = 1; // slices found and not yet added
#pragma unroll 1
    for (int c = c0 + 1;; c += 32) {
        const uint32_t ends = __ballot_sync(0xffffffffu, flags & kHeadEnd);
        const int stop = ends != 0 ? __ffs(ends) - 1 : 31;
        const bool mine = lane <= stop && (flags & kHeadValid);
        bad |= __any_sync(0xffffffffu, mine && (flags & kHeadBad));
        uint32_t valid = __ballot_sync(0xffffffffu, mine);
        const bool over = ends != 0 || c + 32 >= ctas;
        if (!over)
            flags = c + 32 + lane < ctas ? p.records[c + 32 + lane].x : 0;
#pragma unroll 1
        while (valid != 0 || (over && n > 0)) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (i >= n && valid != 0) {
                    slot[i] = 2 * (c + __ffs(valid) - 1);
                    valid &= valid - 1;
                    n = i + 1;
                }
            if (n < kAtOnce && !over)
                break;
            float2 ml[kAtOnce];
            float4 y[kAtOnce][2];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int64_t at = (int64_t)(i < n ? slot[i] : slot[0]) * p.slot_rows + at_row;
                ml[i] = p.part_ml[at];
                y[i][0] = *reinterpret_cast<const float4 *>(p.part_o + at * D + col);
                y[i][1] = *reinterpret_cast<const float4 *>(p.part_o + at * D + col + 4);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (i >= n || ml[i].y == 0.f) // (nothing is seen there; NaN scores leave m at -inf, but l NaN)
                    continue;
                const float top = fmaxf(m, ml[i].x);
                const float w0 = m == -INFINITY ? 0.f : ex2_approx(m - top), w1 = ex2_approx(ml[i].x - top);
                m = top;
                l = l * w0 + ml[i].y * w1;
                const float x[8] = {y[i][0].x, y[i][0].y, y[i][0].z, y[i][0].w,
                                    y[i][1].x, y[i][1].y, y[i][1].z, y[i][1].w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = ta_weighed(o[e], w0) + ta_weighed(x[e], w1);
            }
            n = 0;
        }
        if (over)
            break;
    }
    if (row >= rec.w)
        return;
    const bool zero = bad != 0 || l == 0.f;
    const float inv = 1.f / l;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
        w[e] = zero ? 0u : *reinterpret_cast<const uint32_t *>(&h);
    }
    const int64_t out_row = ((int64_t)rec.y + row / p.group) * p.num_q_heads + rec.z * p.group + row % p.group;
    *reinterpret_cast<uint4 *>(p.out + out_row * D + col) = make_uint4(w[0], w[1], w[2], w[3]);
    if (col == 0 && p.lse != nullptr)
        p.lse[out_row] = zero ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- host side

struct TaEntry {
    int D;
    const void *attn, *combine;
    uint32_t smem;
};

const TaEntry kTaTable[] = {
    {64, reinterpret_cast<const void *>(&tree_attn_kernel<64>), reinterpret_cast<const void *>(&tree_combine_kernel<64>),
     TaCfg<64>::kSmem},
    {128, reinterpret_cast<const void *>(&tree_attn_kernel<128>),
     reinterpret_cast<const void *>(&tree_combine_kernel<128>), TaCfg<128>::kSmem},
    {256, reinterpret_cast<const void *>(&tree_attn_kernel<256>),
     reinterpret_cast<const void *>(&tree_combine_kernel<256>), TaCfg<256>::kSmem},
};

const TaEntry *ta_find(int D)
{
    for (const TaEntry &e : kTaTable)
        if (e.D == D)
            return &e;
    return nullptr;
}

// Once per device: the kernel's shared memory.
bool ta_ready(int device, const TaEntry *e)
{
    constexpr int kDevices = 64;
    static bool done[kDevices][3] = {};
    if (device < 0 || device >= kDevices)
        return false;
    bool &slot = done[device][e - kTaTable];
    if (!slot)
        slot = cudaFuncSetAttribute(e->attn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)e->smem) == cudaSuccess;
    return slot;
}

} // namespace

pkv_status tree_shape(int batch, int total_q, int max_blocks, int num_q_heads, int max_nodes,
                      const pkv_cache_desc *desc, TreeShape *s)
{
    const pkv_status st = check_desc(desc);
    if (st != PKV_OK)
        return st;
    if (batch < 0 || total_q < 0 || max_blocks < 1 || num_q_heads < 1 || max_nodes < 1 ||
        num_q_heads % desc->num_kv_heads != 0)
        return PKV_EINVAL;
    s->group = num_q_heads / desc->num_kv_heads;
    if (batch > kMaxTreeBatch || max_nodes > kTreeMaxNodes || desc->page_size < 8 || s->group > kTaRows ||
        (int64_t)total_q * num_q_heads >= ((int64_t)1 << 31))
        return PKV_EUNSUPPORTED;
    s->q_tile = kTaRows / s->group;
    s->slot_rows = (s->q_tile < max_nodes ? s->q_tile : max_nodes) * s->group;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    s->off_rows = up(kTaMaxCtas * sizeof(int4));
    s->off_ml = s->off_rows + up((size_t)kTaMaxCtas * 4 * kTaRows * sizeof(float2));
    s->off_o = s->off_ml + up((size_t)2 * kTaMaxCtas * s->slot_rows * sizeof(float2));
    s->bytes = 256 + s->off_o + up((size_t)2 * kTaMaxCtas * s->slot_rows * desc->head_dim * sizeof(float));
    return PKV_OK;
}

cudaError_t launch_tree_attn(const TreeArgs &a, cudaStream_t stream)
{
    const TaEntry *e = ta_find(a.desc.head_dim);
    int dev = 0;
    if (e == nullptr || cudaGetDevice(&dev) != cudaSuccess || !ta_ready(dev, e))
        return cudaErrorInvalidValue;
    unsigned char *ws =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(a.workspace) + 255) & ~uintptr_t(255));
    TaParams p;
    p.indptr = a.qo_indptr;
    p.mask = a.tree_mask;
    p.table = a.block_table;
    p.seqlens = a.cache_seqlens;
    p.v_cache = static_cast<const __nv_bfloat16 *>(a.v_cache);
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.err_flag = a.err_flag;
    p.records = reinterpret_cast<int4 *>(ws);
    p.row_ml = reinterpret_cast<float2 *>(ws + a.shape.off_rows);
    p.part_ml = reinterpret_cast<float2 *>(ws + a.shape.off_ml);
    p.part_o = reinterpret_cast<float *>(ws + a.shape.off_o);
    p.batch = a.batch;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.desc.num_kv_heads;
    p.group = a.shape.group;
    p.total_q = a.total_q;
    p.max_blocks = a.max_blocks;
    p.max_nodes = a.max_nodes;
    p.words = a.mask_words;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.desc.page_size)
        ++p.page_shift;
    p.box_shift = p.page_shift < 6 ? p.page_shift : 6;
    p.num_pages = a.desc.num_pages;
    p.layout = a.desc.layout;
    p.q_tile = a.shape.q_tile;
    p.slot_rows = a.shape.slot_rows;
    p.q_scale = a.q_scale;
    p.pdl = a.after_append ? 1 : 0;
    p.pair = a.desc.num_kv_heads % 2 == 0 && a.max_nodes > a.shape.q_tile && sm_count(dev) > 1 ? 1 : 0;
    p.k65536 = 65536u;
    p.wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    const int box_nodes = a.shape.slot_rows / a.shape.group < a.total_q ? a.shape.slot_rows / a.shape.group : a.total_q;
    p.q_box_bytes = (uint32_t)box_nodes * a.shape.group * 128;
    TaMaps m;
    if (!encode_tree_maps(a.desc, a.k_cache, a.v_cache, a.q, a.num_q_heads, a.total_q, a.shape.group, box_nodes, &m.k,
                          &m.v, &m.q))
        return cudaErrorInvalidValue;

    const int grid = sm_count(dev) < kTaMaxCtas ? sm_count(dev) : kTaMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kTaThreads);
    cfg.dynamicSmemBytes = e->smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.pdl ? 1 : 0;
    void *args[] = {&p, &m};
    cudaError_t err = cudaLaunchKernelExC(&cfg, e->attn, args);
    if (err != cudaSuccess)
        return err;
    int ctas = grid;
    const int rows_a_block = kCombineThreads / (a.desc.head_dim / 8);
    cfg.gridDim = dim3(grid, (a.shape.slot_rows + rows_a_block - 1) / rows_a_block);
    cfg.blockDim = dim3(kCombineThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    void *combine_args[] = {&p, &ctas};
    return cudaLaunchKernelExC(&cfg, e->combine, combine_args);
}

} // namespace pkv
