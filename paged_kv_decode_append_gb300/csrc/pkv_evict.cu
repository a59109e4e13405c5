// pkv_evict.cu -- a row's cache cut down to a budget of slots: which slots stay
// (pkv_evict_plan) and the moves that close the gaps (pkv_evict_apply).
//
// Every (layer, row, kv head) keeps as many slots but its own choice of them.
// What is kept behind the budget moves into the holes before it, in order, and
// nothing else moves: attention does not care for the order of the cached
// tokens, and with a few tokens over the budget a compaction that kept the
// order would move nearly all of them.  Sources lie behind the budget, holes
// before it: no move reads what another one writes.
//
// What bounds them.  The plan reads 8 bytes a slot and writes little: 36 layers x 64
// rows x 8 heads of 2,049 .. 2,112 slots (312 MB, 47 us at the copy rate) take 81
// us, 3.9 TB/s.  It is bound by instructions (74 % of the issue slots, 59 % of the
// integer pipe's; 26 for 32 slots in four passes, the rest what a unit does once).
// The moves are memory: half of 8 x 1,000 tokens in 36 layers (609 MB) in 108 us, 5.6
// TB/s, 85 % of the copy rate, rows of 256 bytes from scattered pages.  Small ones:
// 2.9 and 3.6 us.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

// ------------------------------------------------------------------- plan

constexpr int kBins = 256;
constexpr int kPlanList = 128;           // slots that are ranked against one another
constexpr uint32_t kSafeKey = 0xffffffffu; // protected slots: above +inf's key

struct PlanParams {
    const float *mass;
    const int32_t *pos, *seqlens, *evicted, *budgets;
    int2 *moves;
    int32_t *num_moves, *row_lens, *err_flag;
    int batch, num_kv_heads, slots, sink, recent, max_moves;
    int cached; // keys that shared memory holds
};

// What becomes of a row: keep slots of L.
struct PlanRow {
    int L, keep, err;
};
__device__ __forceinline__ PlanRow plan_row(const PlanParams &p, int b)
{
    PlanRow r;
    r.L = p.seqlens[b];
    const int budget = p.budgets[b];
    r.err = 0;
    r.keep = r.L < 0 || budget < 0 ? r.L : min(budget, r.L);
    if (r.L > p.slots || min(r.keep, r.L - r.keep) > p.max_moves) {
        r.err = PKV_ERR_OVERFLOW;
        r.keep = r.L;
    }
    return r;
}

// A mass as a whole number, in the order of floats: NaN below all, -0 as 0.  Never
// kSafeKey.
__device__ __forceinline__ uint32_t plan_rank(uint32_t mass)
{
    const float m = __uint_as_float(mass);
    const uint32_t u = __float_as_uint(m + 0.0f);
    return m != m ? 0u : u ^ (uint32_t)((int32_t)u >> 31 | 0x80000000);
}
constexpr uint32_t kPlainMost = 0x7f800000; // bits of masses 0 .. +inf are their order

// The keys of a (layer, row, kv head), its slots' importance as whole numbers:
// kSafeKey if protected, else by mass.  KEYS of them in every thread's registers,
// slot tid + THREADS k in place k (past the row: kSafeKey); or (KEYS = 0) as many as
// fit in shared memory and the others made anew whenever they are looked at.
template <int THREADS, int KEYS> struct PlanKeys {
    static constexpr int kWarps = THREADS / 32;
    uint32_t k[KEYS > 0 ? KEYS : 1];
    const float *mass;
    const int32_t *pos;
    uint32_t *held; // KEYS > 0: the masses, then the positions
    int L, cached, sink;
    uint32_t open; // positions from sink on that are not protected
    bool crowded;  // KEYS = 0: keys as in crowd

    __device__ __forceinline__ bool safe(int position) const
    {
        return (uint32_t)position - (uint32_t)sink >= open;
    }
    __device__ __forceinline__ uint32_t key(uint32_t rank, int position) const
    {
        if (KEYS == 0 && crowded)
            return safe(position) ? rank + 1 : 0;
        return safe(position) ? kSafeKey : rank;
    }
    __device__ __forceinline__ uint32_t at(int i) const
    {
        if (KEYS > 0)
            return key(held[i], (int)held[KEYS * THREADS + i]);
        return i < cached ? held[i] : key(plan_rank(__float_as_uint(mass[i])), pos[i]);
    }
    // Through shared memory all of a row is under way at once and takes no
    // registers meanwhile (loads into registers, for which the compiler has none to
    // spare and waits one by one, took 10 us).  The whole CTA.
    __device__ __forceinline__ void load(int tid, int slots)
    {
        if (KEYS > 0) {
            uint32_t *held_pos = held + KEYS * THREADS;
            if (slots % 4 == 0) { // every row begins on 16 bytes
                for (int i = 4 * tid; i < L; i += 4 * THREADS) {
                    copy16(held + i, mass + i);
                    copy16(held_pos + i, pos + i);
                }
            } else {
                for (int i = tid; i < L; i += THREADS) {
                    copy4(held + i, mass + i);
                    copy4(held_pos + i, pos + i);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
        } else {
            hold(tid);
        }
    }
    __device__ __forceinline__ void hold(int tid)
    {
        for (int i = tid; i < min(L, cached); i += THREADS)
            held[i] = key(plan_rank(__float_as_uint(mass[i])), pos[i]);
    }
    // Keys into registers.  Masses are taken for their bits, which is right for 0 ..
    // +inf; if there are others their ranks are put in their place first.
    __device__ __forceinline__ void take(int tid)
    {
        if (KEYS > 0)
#pragma unroll
            for (int j = 0; j < KEYS; ++j) { // (there is room for all places; what lies past the row is not looked at)
                const int i = tid + j * THREADS;
                const uint32_t rank = min(held[i], kSafeKey - 1), from = held[KEYS * THREADS + i] - (uint32_t)sink;
                k[j] = (from < open) & (L - tid > j * THREADS) ? rank : kSafeKey;
            }
    }
    __device__ __forceinline__ void rank(int tid)
    {
#pragma unroll 1
        for (int i = tid; i < L; i += THREADS)
            held[i] = plan_rank(held[i]);
    }
    // More slots are protected than stay: they alone are ranked, by mass, above the
    // others, whose key becomes 0.
    __device__ __forceinline__ void crowd(int tid, bool ranked)
    {
        if (KEYS > 0) {
#pragma unroll 1
            for (int i = tid; i < L; i += THREADS) {
                const uint32_t rank = ranked ? held[i] : plan_rank(held[i]);
                held[i] = safe((int)held[KEYS * THREADS + i]) ? rank + 1 : 0;
                held[KEYS * THREADS + i] = (uint32_t)sink; // not protected any more
            }
            open = 1;
        } else {
            crowded = true;
            hold(tid);
        }
    }
    static __device__ __forceinline__ void copy16(void *to, const void *from)
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
    }
    static __device__ __forceinline__ void copy4(void *to, const void *from)
    {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(to)), "l"(from) : "memory");
    }
    // f(slot, key) for the slots of this thread, and for the places past the row
    template <typename F> __device__ __forceinline__ void each(int tid, F f) const
    {
        if (KEYS > 0) {
#pragma unroll
            for (int j = 0; j < KEYS; ++j)
                f(tid + j * THREADS, k[j]);
        } else {
            for (int i = tid; i < L; i += THREADS)
                f(i, at(i));
        }
    }
    // the same one by one, in less code
    template <typename F> __device__ __forceinline__ void each_rarely(int tid, F f) const
    {
#pragma unroll 1
        for (int i = tid; i < L; i += THREADS)
            f(i, at(i));
    }
    // A bit for every slot that f(slot, key) says, 32 slots a word.  The whole CTA.
    template <typename F> __device__ __forceinline__ void mark(int tid, uint32_t *bits, F f) const
    {
        const int lane = tid & 31;
        if (KEYS > 0) {
#pragma unroll
            for (int j = 0; j < KEYS; ++j) {
                const uint32_t word = __ballot_sync(0xffffffffu, f(tid + j * THREADS, k[j]));
                if (lane == 0) // (there is room for all places)
                    bits[(tid >> 5) + j * kWarps] = word;
            }
        } else {
            for (int i = tid; (i & ~31) < L; i += THREADS) {
                const uint32_t word = __ballot_sync(0xffffffffu, i < L && f(i, at(i)));
                if (lane == 0)
                    bits[i >> 5] = word;
            }
        }
    }
};

// One more in the bin of x = key - from, if that is in the open range.  Without a
// branch: there are many and most are in range or most are not.
__device__ __forceinline__ void plan_count(uint32_t bins, uint32_t x, uint32_t width, int shift)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.le.u32 p, %0, %1;\n\t"
                 "@p red.shared.add.u32 [%2], 1;\n\t}" ::"r"(x),
                 "r"(width), "r"(bins + ((x >> shift) << 2))
                 : "memory");
}
// Appends (key, ~slot) to the list, if x = key - from is below `size`.
__device__ __forceinline__ void plan_append(uint32_t count, uint32_t list, uint32_t x, uint32_t size, uint32_t key, int i)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .u32 n;\n\t"
                 "setp.lt.u32 p, %0, %1;\n\t"
                 "@p atom.shared.add.u32 n, [%2], 1;\n\t"
                 "@p mad.lo.u32 n, n, 8, %3;\n\t"
                 "@p st.shared.v2.u32 [n], {%4, %5};\n\t}" ::"r"(x),
                 "r"(size), "r"(count), "r"(list), "r"(~(uint32_t)i), "r"(key)
                 : "memory");
}

// One CTA for each (layer, row, kv head).  Slots are ranked by key (protected ones
// first; where those are too many, among themselves by mass), equal keys
// by slot, the lowest first.  The key of the last slot that stays is found by
// counting into 256 bins over the range that is still open, narrowed until a bin
// is to be taken whole or has at most 128 slots, which are ranked against one
// another.  Masses of a row spread over many powers of two and a float's bits
// are its logarithm, so that the first count nearly always does.  Where more
// slots than that have one and the same key, the count goes on over the slots.
// Few threads with many keys each: what a warp does once (votes, scans, waits)
// then weighs less.
template <int THREADS, int KEYS>
__global__ void __launch_bounds__(THREADS, (KEYS == 0 ? 1024 : 1280) / THREADS)
    evict_plan_kernel(const __grid_constant__ PlanParams p)
{
    constexpr int kWarps = THREADS / 32;
    extern __shared__ __align__(16) uint32_t s_dyn[]; // keys (or what they are made from), a bit for every slot that stays
    __shared__ __align__(16) int s_bins[kBins];
    __shared__ uint64_t s_list[kPlanList];
    __shared__ int2 s_scan[kWarps];
    __shared__ uint32_t s_lo, s_hi;
    __shared__ int s_safe, s_count, s_k, s_in;
    __shared__ uint32_t s_from;
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t unit = blockIdx.x;
    const int per_layer = p.batch * p.num_kv_heads;
    const int layer = (int)(blockIdx.x / (unsigned)per_layer), rest = (int)(blockIdx.x - (unsigned)(layer * per_layer));
    const int b = rest / p.num_kv_heads, g = rest - b * p.num_kv_heads;
    const int gone = p.evicted != nullptr ? p.evicted[b] : 0;
    const PlanRow r = plan_row(p, b);
    const int64_t oldest = (int64_t)r.L + gone - p.recent - 1; // position before the newest `recent` ones
    if (tid == 0) {
        if (layer == 0 && g == 0) {
            p.row_lens[2 * b] = r.L;
            p.row_lens[2 * b + 1] = r.keep;
            set_error(p.err_flag, r.err);
        }
        if (r.keep >= r.L || r.keep == 0)
            p.num_moves[unit] = 0;
        s_lo = kSafeKey;
        s_hi = 0;
        s_safe = s_count = 0;
    }
    if (r.keep >= r.L || r.keep == 0)
        return;
    const int L = r.L, keep = r.keep, words = (L + 31) / 32;
    uint32_t *bits = s_dyn + (KEYS > 0 ? 2 * KEYS * THREADS : p.cached);
    PlanKeys<THREADS, KEYS> keys;
    keys.mass = p.mass + unit * p.slots;
    keys.pos = p.pos + unit * p.slots;
    keys.held = s_dyn;
    keys.L = L;
    keys.cached = p.cached;
    keys.sink = p.sink;
    keys.crowded = false;
    keys.open = (uint32_t)(max((int64_t)p.sink - 1, min((int64_t)INT32_MAX, oldest)) - p.sink + 1);
    keys.load(tid, p.slots);
    auto no_bins = [&] {
        for (int i = tid; i < kBins / 4; i += THREADS)
            reinterpret_cast<int4 *>(s_bins)[i] = make_int4(0, 0, 0, 0);
    };
    no_bins();
    __syncthreads();

    // Protected slots, and the range of the others' keys.
    int safe;
    for (bool ranked = KEYS == 0, crowded = false;;) {
        keys.take(tid);
        uint32_t lo = kSafeKey, hi = 0;
        safe = 0;
        keys.each(tid, [&](int, uint32_t k) {
            safe += k == kSafeKey ? 1 : 0;
            lo = min(lo, k);     // (a protected slot's key changes nothing)
            hi = max(hi, k + 1); // (that of a protected slot becomes 0)
        });
        safe = __reduce_add_sync(0xffffffffu, safe);
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            atomicAdd(&s_safe, safe);
            atomicMin(&s_lo, lo);
            atomicMax(&s_hi, hi);
        }
        __syncthreads();
        safe = s_safe - (KEYS > 0 ? KEYS * THREADS - L : 0);
        const bool plain = ranked || s_hi <= kPlainMost + 1;
        if (plain && (safe <= keep || crowded))
            break;
        __syncthreads();
        if (!plain) {
            keys.rank(tid); // negative masses, -0 or NaN
        } else {
            keys.crowd(tid, ranked);
            crowded = true;
        }
        ranked = true;
        if (tid == 0) {
            s_lo = kSafeKey;
            s_hi = 0;
            s_safe = 0;
        }
        __syncthreads();
    }

    // The open range [from, from + width]: of keys, or (`among`) of ~slot among the
    // slots of key `tie`.
    uint32_t from = s_lo, width = s_hi - 1 - s_lo, tie = 0;
    int k = keep - safe, in = L - safe; // the k-th greatest of `in` slots there is looked for
    bool among = keep == safe;
    auto ties = [&](uint32_t key) {
        among = true;
        tie = key;
        from = ~(uint32_t)(L - 1);
        width = L - 1;
    };
    if (among) {
        ties(kSafeKey);
        k = keep;
        in = safe;
    }
    // (A round leaves a 256th of the range: at most four of keys and four of slots.)
    for (int round = 0; round < 8 && in > kPlanList && k < in; ++round) {
        if (!among && width == 0)
            ties(from);
        const int shift = max(0, 24 - __clz(width)); // 256 bins over the range
        if (among)
            keys.each_rarely(tid, [&](int i, uint32_t key) {
                if (key == tie && ~(uint32_t)i - from <= width)
                    atomicAdd(&s_bins[(~(uint32_t)i - from) >> shift], 1);
            });
        else
            keys.each(tid, [&](int, uint32_t key) { plan_count(smem_addr(s_bins), key - from, width, shift); });
        __syncthreads();
        if (warp == 0) { // from the top: a lane holds 8 bins
            const int4 *at = reinterpret_cast<const int4 *>(s_bins) + 2 * (31 - lane);
            const int4 x = at[0], y = at[1];
            const int n[8] = {y.w, y.z, y.y, y.x, x.w, x.z, x.y, x.x};
            const int sum = (n[0] + n[1]) + (n[2] + n[3]) + (n[4] + n[5]) + (n[6] + n[7]);
            int before = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, before, d);
                before += lane >= d ? up : 0;
            }
            before -= sum;
            if (before < k && before + sum >= k) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (before < k && before + n[j] >= k) {
                        s_from = (uint32_t)(kBins - 1 - (8 * lane + j)) << shift;
                        s_k = k - before;
                        s_in = n[j];
                    }
                    before += n[j];
                }
            }
        }
        __syncthreads();
        width = min(width - s_from, (1u << shift) - 1);
        from += s_from;
        k = s_k;
        in = s_in;
        if (in > kPlanList && k < in) { // once more
            no_bins();
            __syncthreads();
        }
    }
    // A bit for every slot that stays: those above the open range, and of those in
    // it the k first, unless all do.
    const bool all = k == in;
    // (Keys that are made anew for every pass could change under a writer that does
    // not belong there; nothing goes past its array even then.)
    in = min(in, kPlanList);
    auto list_late = [&](uint32_t key, int i) {
        const int n = atomicAdd(&s_count, 1);
        if (n < kPlanList)
            s_list[n] = (uint64_t)key << 32 | ~(uint32_t)i;
    };
    if (among) { // key `tie`: up to slot `last`
        int last = (int)~from;
        if (!all) {
            keys.each_rarely(tid, [&](int i, uint32_t key) {
                if (key == tie && ~(uint32_t)i - from <= width)
                    list_late(0, i);
            });
            __syncthreads();
            if (tid < in) {
                const uint64_t x = s_list[tid];
                int above = 0;
                for (int j = 0; j < in; ++j)
                    above += s_list[j] > x ? 1 : 0;
                if (above == k - 1)
                    s_last = (int)~(uint32_t)x;
            }
            __syncthreads();
            last = s_last;
        }
        keys.mark(tid, bits, [&](int i, uint32_t key) { return (key > tie) | ((key == tie) & (i <= last)); });
    } else {
        const uint32_t size = all ? 0 : width + 1, stays = from + size;
        keys.mark(tid, bits, [&](int i, uint32_t key) {
            if (KEYS > 0)
                plan_append(smem_addr(&s_count), smem_addr(s_list), key - from, size, key, i);
            else if (key - from < size)
                list_late(key, i);
            return key >= stays;
        });
        if (!all) {
            __syncthreads();
            if (tid < in) { // (at most 128)
                const uint64_t x = s_list[tid];
                int above = 0;
                for (int j = 0; j < in; ++j)
                    above += s_list[j] > x ? 1 : 0;
                const uint32_t i = ~(uint32_t)x;
                if (above < k && (KEYS > 0 || i < (uint32_t)L))
                    atomicOr(&bits[i >> 5], 1u << (i & 31));
            }
        }
    }
    __syncthreads();

    // Holes before the budget and slots that stay behind it, i-th to i-th: how many
    // there are before every word, then the words' bits.
    auto holes_of = [&](int w) {
        const int n = keep - w * 32; // (below L)
        return n <= 0 ? 0u : ~bits[w] & (n >= 32 ? 0xffffffffu : (1u << n) - 1);
    };
    auto extra_of = [&](int w) {
        const int n = keep - w * 32, e = L - w * 32;
        const uint32_t word = bits[w] & (e >= 32 ? 0xffffffffu : (1u << e) - 1); // of the row's slots
        return n <= 0 ? word : n >= 32 ? 0u : word & ~((1u << n) - 1);
    };
    int2 *out = p.moves + unit * p.max_moves;
    if (KEYS > 0) {
        // A word a thread (there are fewer), its holes or what stays behind the budget;
        // the word that the budget cuts has both, and its holes come last.  Both counts
        // in one number; the list is put together where the masses were.
        const int cut = keep >> 5, w = tid == words ? cut : tid;
        const bool hole = tid < cut || tid == words;
        const uint32_t word = tid > words ? 0 : hole ? holes_of(w) : extra_of(w);
        const uint32_t bits_of = (uint32_t)__popc(word), mine = hole ? bits_of : bits_of << 16;
        uint32_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, upto, d);
            upto += lane >= d ? x : 0;
        }
        if (lane == 31)
            s_scan[warp].x = (int)upto;
        __syncthreads();
        uint32_t before = upto - mine, total = 0;
#pragma unroll
        for (int i = 0; i < KEYS * kWarps / 32 + 1; ++i) { // warps that have words
            before += i < warp ? (uint32_t)s_scan[i].x : 0;
            total += (uint32_t)s_scan[i].x;
        }
        int *list = reinterpret_cast<int *>(s_dyn);
        uint32_t at = hole ? 2 * (before & 0xffff) + 1 : 2 * (before >> 16);
        // A few words of many bits the warp does together, one after the other: rows of
        // 2,112 slots that keep 2,048 take 86 us with every word a thread's, 80 so; where
        // most words have many bits (1,056 kept) all of them so take 137, none 115, and up
        // to twelve of a warp 111.
        uint32_t dense = __ballot_sync(0xffffffffu, bits_of > 4);
        dense = __popc(dense) > 12 ? 0 : dense;
        for (uint32_t m = dense; m != 0; m &= m - 1) {
            const int from = __ffs(m) - 1;
            const uint32_t of = __shfl_sync(0xffffffffu, word, from), to = __shfl_sync(0xffffffffu, at, from);
            const int slot = __shfl_sync(0xffffffffu, w, from) * 32 + lane;
            if ((of >> lane & 1) != 0)
                list[to + 2 * __popc(of & ((1u << lane) - 1))] = slot;
        }
        for (uint32_t m = (dense >> lane & 1) != 0 ? 0 : word; m != 0; m &= m - 1, at += 2)
            list[at] = w * 32 + __ffs(m) - 1;
        __syncthreads();
        const int n = (int)(total >> 16);
        for (int i = tid; i < n; i += THREADS)
            out[i] = reinterpret_cast<const int2 *>(list)[i];
        if (tid == 0)
            p.num_moves[unit] = n;
    } else {
        const int per_thread = (words + THREADS - 1) / THREADS;
        const int a = min(words, tid * per_thread), z = min(words, a + per_thread);
        int2 mine = make_int2(0, 0);
        for (int w = a; w < z; ++w) {
            mine.x += __popc(extra_of(w));
            mine.y += __popc(holes_of(w));
        }
        int2 upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto.x, d), y = __shfl_up_sync(0xffffffffu, upto.y, d);
            upto.x += lane >= d ? x : 0;
            upto.y += lane >= d ? y : 0;
        }
        if (lane == 31)
            s_scan[warp] = upto;
        __syncthreads();
        int2 at = make_int2(upto.x - mine.x, upto.y - mine.y);
        for (int w = 0; w < warp; ++w) {
            at.x += s_scan[w].x;
            at.y += s_scan[w].y;
        }
        for (int w = a; w < z; ++w) {
            for (uint32_t m = extra_of(w); m != 0 && at.x < p.max_moves; m &= m - 1)
                out[at.x++].x = w * 32 + __ffs(m) - 1;
            for (uint32_t m = holes_of(w); m != 0 && at.y < p.max_moves; m &= m - 1)
                out[at.y++].y = w * 32 + __ffs(m) - 1;
        }
        if (tid == THREADS - 1)
            p.num_moves[unit] = min(at.x, p.max_moves);
    }
}

// ------------------------------------------------------------------- apply

constexpr int kApplyThreads = 256;
constexpr int kApplyChunk = 128; // moves whose addresses are worked out together
constexpr int kApplyAhead = 4;   // 16-byte pieces of a thread under way at once
constexpr int kApplyLayers = 128;

struct ApplyParams {
    void *k[kApplyLayers], *v[kApplyLayers];
    const int2 *moves;
    const int32_t *num_moves, *row_lens, *table;
    float *mass;
    int32_t *pos;
    int32_t *seqlens, *evicted, *err_flag;
    int batch, max_moves, max_blocks, page_shift, num_pages, num_kv_heads, head_dim, layout, slots;
};

// blockIdx.x: (layer, row, kv head); blockIdx.y: its chunks of moves, dealt out in turn.
__global__ void __launch_bounds__(kApplyThreads) evict_apply_kernel(const __grid_constant__ ApplyParams p)
{
    __shared__ int64_t s_src[kApplyChunk], s_dst[kApplyChunk];
    const int tid = threadIdx.x;
    const int64_t unit = blockIdx.x;
    const int per_layer = p.batch * p.num_kv_heads;
    const int layer = (int)(unit / per_layer), rest = (int)(unit - (int64_t)layer * per_layer);
    const int b = rest / p.num_kv_heads, g = rest - b * p.num_kv_heads;
    const int n = p.num_moves[unit];
    const int before = p.row_lens[2 * b], after = p.row_lens[2 * b + 1];
    const bool first = blockIdx.y == 0;
    const bool leads = first && layer == 0 && g == 0; // keeps the row's lengths
    if (before < 0 || after < 0 || (n == 0 && !leads) || (!first && (int64_t)blockIdx.y * kApplyChunk >= n))
        return;
    const int32_t *row = p.table + (int64_t)b * p.max_blocks;
    const int2 *moves = p.moves + unit * p.max_moves;
    int err = 0;
    if (after > before)
        err = PKV_ERR_MOVE;
    else if (before > (int64_t)p.max_blocks << p.page_shift ||
             (before > p.slots && (p.mass != nullptr || p.pos != nullptr)))
        err = PKV_ERR_OVERFLOW;
    if (err == 0) { // all of the row's pages: its units go together
        const int pages = (int)(((int64_t)before + (1 << p.page_shift) - 1) >> p.page_shift);
        for (int i = tid; i < pages; i += kApplyThreads)
            if (row[i] < 1 || row[i] >= p.num_pages)
                err = PKV_ERR_PAGE;
    }
    if (err != 0)
        set_error(p.err_flag, err);
    if (__syncthreads_or(err))
        return;
    if (leads && tid == 0 && p.seqlens != nullptr) {
        if (p.evicted != nullptr)
            p.evicted[b] += p.seqlens[b] - after;
        p.seqlens[b] = after;
    }
    if (n < 0 || n > p.max_moves) {
        if (tid == 0)
            set_error(p.err_flag, PKV_ERR_MOVE);
        return;
    }
    const int D = p.head_dim, per_row = D / 8;
    const int64_t P = (int64_t)1 << p.page_shift;
    auto element = [&](int slot) {
        const int64_t page = row[slot >> p.page_shift], at = slot & (P - 1);
        return p.layout == PKV_NHD ? ((page * P + at) * p.num_kv_heads + g) * D
                                   : ((page * p.num_kv_heads + g) * P + at) * D;
    };
    uint4 *kp = static_cast<uint4 *>(p.k[layer]), *vp = static_cast<uint4 *>(p.v[layer]);
    for (int c = blockIdx.y * kApplyChunk; c < n; c += gridDim.y * kApplyChunk) {
        const int m = min(kApplyChunk, n - c);
        __syncthreads();
        if (tid < m) {
            const int2 mv = moves[c + tid];
            // a source behind the slots that stay, a hole among them: no two moves meet
            const bool good = mv.x >= after && mv.x < before && mv.y >= 0 && mv.y < after;
            if (!good)
                set_error(p.err_flag, PKV_ERR_MOVE);
            s_src[tid] = good ? element(mv.x) / 8 : -1;
            s_dst[tid] = good ? element(mv.y) / 8 : -1;
            if (good && p.mass != nullptr)
                p.mass[unit * p.slots + mv.y] = p.mass[unit * p.slots + mv.x];
            if (good && p.pos != nullptr)
                p.pos[unit * p.slots + mv.y] = p.pos[unit * p.slots + mv.x];
        }
        __syncthreads();
        // a K row, then its V row, 16 bytes a thread
        const int pieces = 2 * per_row * m;
        for (int x0 = tid; x0 < pieces; x0 += kApplyThreads * kApplyAhead) {
            uint4 d[kApplyAhead];
            uint4 *to[kApplyAhead];
#pragma unroll
            for (int u = 0; u < kApplyAhead; ++u) {
                const int x = x0 + u * kApplyThreads, i = x / (2 * per_row), e = x - i * 2 * per_row;
                to[u] = nullptr;
                if (x < pieces && s_src[i] >= 0) {
                    uint4 *pool = e < per_row ? kp : vp;
                    const int piece = e < per_row ? e : e - per_row;
                    d[u] = pool[s_src[i] + piece];
                    to[u] = pool + s_dst[i] + piece;
                }
            }
#pragma unroll
            for (int u = 0; u < kApplyAhead; ++u)
                if (to[u] != nullptr)
                    *to[u] = d[u];
        }
    }
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}
bool aligned4(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}
bool aligned8(const void *p) // moves are read and written in pairs
{
    return (reinterpret_cast<uintptr_t>(p) & 7u) == 0;
}

constexpr int kPlanCached = 38912; // keys in shared memory at most; longer rows make theirs again

// Keys in registers up to 17,408 slots, 17 a thread at most, then in shared memory.
// As few threads as that allows: 36 x 64 x 8 rows of 1,100 slots take 62 us with nine
// keys in each of 128 threads, 81 with 17 of which half are idle, 116 with nine in 256;
// of 2,112 slots 81 with 17 in 128, 113 with nine in 256; of 3,900 218 with 17 in 256
// (31 in 128, which registers still hold, 215).  36 x 16 x 8 of 8,192: 134 with 17 in
// 512, 233 with keys in shared memory; 36 x 8 x 8 of 16,384: 169 with 17 in 1,024, 288
// with keys in shared memory.  Longer ones: 36 x 4 x 8 of 32,000 246 with 1,024
// threads, 305 with 512, 756 with 128.
struct PlanEntry {
    int slots, threads;
    const void *kernel;
};
template <int THREADS, int KEYS> constexpr PlanEntry plan_entry()
{
    return {KEYS > 0 ? THREADS * KEYS : kEvictMaxSlots, THREADS,
            reinterpret_cast<const void *>(&evict_plan_kernel<THREADS, KEYS>)};
}
const PlanEntry kPlanTable[] = {
    plan_entry<128, 1>(),  plan_entry<128, 4>(),  plan_entry<128, 9>(),  plan_entry<128, 17>(),
    plan_entry<256, 17>(), plan_entry<512, 17>(), plan_entry<1024, 17>(), plan_entry<1024, 0>(),
};
constexpr int kPlanEntries = 8, kPlanLong = kPlanEntries - 1; // the last of them

size_t plan_smem(const PlanEntry &e, int slots, int cached)
{
    const bool is_long = &e == &kPlanTable[kPlanLong];
    const size_t held = is_long ? (size_t)cached : 2 * (size_t)e.slots;
    const size_t words = is_long ? ((size_t)slots + 31) / 32 : (size_t)e.slots / 32;
    return (held + words) * sizeof(uint32_t);
}

// Once per device: the shared memory of the kernels that take more than the default.
bool plan_ready(int device)
{
    constexpr int kDevices = 64;
    static bool done[kDevices] = {};
    if (device < 0 || device >= kDevices)
        return false;
    if (!done[device]) {
        bool good = true;
        for (const PlanEntry &e : kPlanTable)
            good = good && cudaFuncSetAttribute(e.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)plan_smem(e, e.slots, kPlanCached)) == cudaSuccess;
        done[device] = good;
    }
    return done[device];
}

} // namespace
} // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_evict_plan(const float *mass, const int32_t *slot_pos, int32_t num_layers, int32_t batch,
                          int32_t num_kv_heads, int32_t slots, const int32_t *cache_seqlens, const int32_t *evicted,
                          const int32_t *budgets, int32_t sink, int32_t recent, int32_t *moves, int32_t max_moves,
                          int32_t *num_moves, int32_t *row_lens, int32_t *err_flag, void *stream)
{
    if (num_layers < 1 || batch < 0 || num_kv_heads < 1 || slots < 1 || sink < 0 || recent < 0 || max_moves < 1)
        return PKV_EINVAL;
    const int64_t units = (int64_t)num_layers * batch * num_kv_heads;
    if (units > 0x7fffffff || slots > kEvictMaxSlots)
        return PKV_EUNSUPPORTED;
    if (batch == 0)
        return PKV_OK;
    if (mass == nullptr || slot_pos == nullptr || cache_seqlens == nullptr || budgets == nullptr || moves == nullptr ||
        num_moves == nullptr || row_lens == nullptr || !slots_aligned(mass, slots) || !slots_aligned(slot_pos, slots) ||
        !aligned8(moves))
        return PKV_EINVAL;
    PlanParams p;
    p.mass = mass;
    p.pos = slot_pos;
    p.seqlens = cache_seqlens;
    p.evicted = evicted;
    p.budgets = budgets;
    p.moves = reinterpret_cast<int2 *>(moves);
    p.num_moves = num_moves;
    p.row_lens = row_lens;
    p.err_flag = err_flag;
    p.batch = batch;
    p.num_kv_heads = num_kv_heads;
    p.slots = slots;
    p.sink = sink;
    p.recent = recent;
    p.max_moves = max_moves;
    const PlanEntry *e = kPlanTable;
    while (slots > e->slots)
        ++e;
    p.cached = slots < kPlanCached ? slots : kPlanCached;
    const size_t smem = plan_smem(*e, slots, p.cached);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !plan_ready(dev))
        return PKV_ECUDA;
    void *args[] = {&p};
    return cudaLaunchKernel(e->kernel, dim3((unsigned)units), dim3(e->threads), args, smem,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ECUDA;
}

pkv_status pkv_evict_apply(const pkv_cache_desc *desc, int32_t num_layers, void *const *k_caches,
                           void *const *v_caches, const int32_t *moves, int32_t max_moves, const int32_t *num_moves,
                           const int32_t *row_lens, const int32_t *block_table, int32_t max_blocks, float *mass,
                           int32_t *slot_pos, int32_t slots, int32_t *cache_seqlens, int32_t *evicted, int32_t batch,
                           int32_t *err_flag, void *stream)
{
    const pkv_status st = check_desc(desc);
    if (st != PKV_OK)
        return st;
    if (num_layers < 1 || max_moves < 1 || max_blocks < 1 || slots < 1 || batch < 0)
        return PKV_EINVAL;
    const int64_t units = (int64_t)num_layers * batch * desc->num_kv_heads;
    if (num_layers > kApplyLayers || units > 0x7fffffff)
        return PKV_EUNSUPPORTED;
    if (k_caches == nullptr || v_caches == nullptr)
        return PKV_EINVAL;
    ApplyParams p;
    for (int l = 0; l < num_layers; ++l) {
        p.k[l] = k_caches[l];
        p.v[l] = v_caches[l];
        if (p.k[l] == nullptr || p.v[l] == nullptr || !aligned16(p.k[l]) || !aligned16(p.v[l]))
            return PKV_EINVAL;
    }
    if (batch == 0)
        return PKV_OK;
    if (moves == nullptr || num_moves == nullptr || row_lens == nullptr || block_table == nullptr || !aligned8(moves) ||
        (cache_seqlens == nullptr && evicted != nullptr) || !aligned4(mass) || !aligned4(slot_pos))
        return PKV_EINVAL;
    p.moves = reinterpret_cast<const int2 *>(moves);
    p.num_moves = num_moves;
    p.row_lens = row_lens;
    p.table = block_table;
    p.mass = mass;
    p.pos = slot_pos;
    p.seqlens = cache_seqlens;
    p.evicted = evicted;
    p.err_flag = err_flag;
    p.batch = batch;
    p.max_moves = max_moves;
    p.max_blocks = max_blocks;
    p.page_shift = 0;
    while ((1 << p.page_shift) < desc->page_size)
        ++p.page_shift;
    p.num_pages = desc->num_pages;
    p.num_kv_heads = desc->num_kv_heads;
    p.head_dim = desc->head_dim;
    p.layout = desc->layout;
    p.slots = slots;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return PKV_ECUDA;
    // a unit's moves over several CTAs where the units alone do not fill the device
    const int64_t most = (max_moves + kApplyChunk - 1) / kApplyChunk, fill = 8 * (int64_t)sm_count(dev);
    int64_t split = (fill + units - 1) / units;
    split = split < most ? split : most;
    split = split < 65535 ? split : 65535;
    evict_apply_kernel<<<dim3((unsigned)units, (unsigned)split), kApplyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

} // extern "C"
