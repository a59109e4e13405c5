// pkv_evict.cu -- a row's cache cut down to a budget of slots: which slots stay
// (pkv_evict_plan) and the moves that close the gaps (pkv_evict_apply).
//
// Every (layer, row, kv head) keeps as many slots but its own choice of them.
// What is kept behind the budget moves into the holes before it, in order, and
// nothing else moves: attention does not care for the order of the cached
// tokens, and with a few tokens over the budget a compaction that kept the
// order would move nearly all of them.  Sources lie behind the budget, holes
// before it: no move reads what another one writes.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

// ------------------------------------------------------------------- plan

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kBins = 256;
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
    if (r.keep < r.L && (r.L > p.slots || min(r.keep, r.L - r.keep) > p.max_moves)) {
        r.err = PKV_ERR_OVERFLOW;
        r.keep = r.L;
    }
    return r;
}

// Importance of a slot as a whole number: protected above all, then by mass
// (NaN below all), the order of floats.
__device__ __forceinline__ uint32_t plan_key(float mass, int pos, int sink, int64_t recent_from)
{
    const uint32_t u = __float_as_uint(mass + 0.0f); // -0 counts as 0
    const uint32_t k = mass != mass ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
    return pos < sink || pos >= recent_from ? kSafeKey : k;
}

__device__ __forceinline__ int plan_sum(int x, int *scratch, int tid)
{
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((tid & 31) == 0)
        scratch[tid >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w)
        x += scratch[w];
    return x;
}

// One CTA for each (layer, row, kv head).
__global__ void __launch_bounds__(kPlanThreads) evict_plan_kernel(const __grid_constant__ PlanParams p)
{
    extern __shared__ uint32_t s_dyn[]; // keys, then a bit for every slot that stays
    __shared__ int s_bins[kBins];
    __shared__ int s_scratch[kPlanWarps];
    __shared__ int2 s_scan[kPlanWarps];
    __shared__ uint32_t s_lo, s_hi;
    __shared__ int s_k, s_all;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t unit = blockIdx.x;
    const int per_layer = p.batch * p.num_kv_heads;
    const int layer = (int)(unit / per_layer), rest = (int)(unit - (int64_t)layer * per_layer);
    const int b = rest / p.num_kv_heads, g = rest - b * p.num_kv_heads;
    const PlanRow r = plan_row(p, b);
    if (tid == 0) {
        if (layer == 0 && g == 0) {
            p.row_lens[2 * b] = r.L;
            p.row_lens[2 * b + 1] = r.keep;
            set_error(p.err_flag, r.err);
        }
        if (r.keep >= r.L || r.keep == 0)
            p.num_moves[unit] = 0;
    }
    if (r.keep >= r.L || r.keep == 0)
        return;
    const int L = r.L, keep = r.keep;
    const float *mass = p.mass + unit * p.slots;
    const int32_t *pos = p.pos + unit * p.slots;
    const int64_t recent_from = (int64_t)L + (p.evicted != nullptr ? p.evicted[b] : 0) - p.recent;
    const bool held = L <= p.cached;
    uint32_t *keys = s_dyn, *bits = s_dyn + p.cached;
    auto key_at = [&](int i) { return held ? keys[i] : plan_key(mass[i], pos[i], p.sink, recent_from); };

    // Protected slots, and the range of the others' keys.
    uint32_t lo = kSafeKey, hi = 0;
    int safe = 0;
    for (int i = tid; i < L; i += kPlanThreads) {
        const uint32_t k = plan_key(mass[i], pos[i], p.sink, recent_from);
        if (held)
            keys[i] = k;
        if (k == kSafeKey) {
            ++safe;
        } else {
            lo = min(lo, k);
            hi = max(hi, k);
        }
    }
    if (tid == 0) {
        s_lo = kSafeKey;
        s_hi = 0;
    }
    safe = plan_sum(safe, s_scratch, tid);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        atomicMin(&s_lo, lo);
        atomicMax(&s_hi, hi);
    }
    __syncthreads();
    lo = s_lo;
    hi = s_hi;

    // The least key that stays, `least`: with `all`, every slot of that key or
    // above; otherwise every one above and the first `ties` of that key.
    uint32_t least;
    int ties = 0;
    bool all = false;
    if (keep <= safe) {
        least = kSafeKey;
        ties = keep;
        all = keep == safe;
    } else {
        int k = keep - safe; // the k-th greatest key of [lo, hi] is looked for
        for (;;) {
            if (lo == hi) {
                least = lo;
                ties = k;
                break;
            }
            const int shift = max(0, 24 - __clz(hi - lo)); // 256 bins over the range
            for (int i = tid; i < kBins; i += kPlanThreads)
                s_bins[i] = 0;
            __syncthreads();
            for (int i = tid; i < L; i += kPlanThreads) {
                const uint32_t x = key_at(i);
                if (x >= lo && x <= hi)
                    atomicAdd(&s_bins[(x - lo) >> shift], 1);
            }
            __syncthreads();
            if (warp == 0) { // from the top: a lane holds 8 bins
                int n[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    n[j] = s_bins[kBins - 1 - (8 * lane + j)];
                    sum += n[j];
                }
                int before = sum;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int up = __shfl_up_sync(0xffffffffu, before, d);
                    before += lane >= d ? up : 0;
                }
                before -= sum;
                if (before < k && before + sum >= k) {
                    int j = 0;
                    while (before + n[j] < k)
                        before += n[j++];
                    const uint32_t bin = kBins - 1 - (8 * lane + j);
                    s_k = k - before;
                    s_all = k - before == n[j];
                    const uint32_t from = lo + (bin << shift);
                    s_lo = from;
                    s_hi = from + min(hi - from, (1u << shift) - 1);
                }
            }
            __syncthreads();
            lo = s_lo;
            hi = s_hi;
            k = s_k;
            all = s_all != 0;
            if (all) {
                least = lo;
                break;
            }
        }
    }

    // A bit for every slot that stays.
    const int words = (L + 31) / 32, per_warp = (words + kPlanWarps - 1) / kPlanWarps;
    const int w0 = warp * per_warp, w1 = min(words, w0 + per_warp);
    int tied = 0; // slots of the least key before this warp's
    if (!all) {
        for (int w = w0; w < w1; ++w) {
            const int i = w * 32 + lane;
            tied += __popc(__ballot_sync(0xffffffffu, i < L && key_at(i) == least));
        }
        __syncthreads();
        if (lane == 0)
            s_scratch[warp] = tied;
        __syncthreads();
        tied = 0;
        for (int w = 0; w < warp; ++w)
            tied += s_scratch[w];
    }
    for (int w = w0; w < w1; ++w) {
        const int i = w * 32 + lane;
        const uint32_t k = i < L ? key_at(i) : 0;
        uint32_t stay = __ballot_sync(0xffffffffu, i < L && (all ? k >= least : k > least));
        if (!all) {
            const uint32_t same = __ballot_sync(0xffffffffu, i < L && k == least);
            stay |= __ballot_sync(0xffffffffu, (same >> lane & 1) && tied + __popc(same & ((1u << lane) - 1)) < ties);
            tied += __popc(same);
        }
        if (lane == 0)
            bits[w] = stay;
    }
    __syncthreads();

    // Holes before the budget and slots that stay behind it, i-th to i-th.
    const int per_thread = (words + kPlanThreads - 1) / kPlanThreads;
    const int a = min(words, tid * per_thread), z = min(words, a + per_thread);
    auto holes_of = [&](int w) {
        const int n = keep - w * 32;
        return n <= 0 ? 0u : ~bits[w] & (n >= 32 ? 0xffffffffu : (1u << n) - 1);
    };
    auto extra_of = [&](int w) {
        const int n = keep - w * 32;
        return n <= 0 ? bits[w] : n >= 32 ? 0u : bits[w] & ~((1u << n) - 1);
    };
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
    int32_t *out = reinterpret_cast<int32_t *>(p.moves + unit * p.max_moves);
    for (int w = a; w < z; ++w) {
        for (uint32_t m = extra_of(w); m != 0; m &= m - 1)
            out[2 * at.x++] = w * 32 + __ffs(m) - 1;
        for (uint32_t m = holes_of(w); m != 0; m &= m - 1)
            out[2 * at.y++ + 1] = w * 32 + __ffs(m) - 1;
    }
    if (tid == kPlanThreads - 1)
        p.num_moves[unit] = at.x;
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
    if (before < 0 || after < 0 || (n == 0 && !(first && layer == 0 && g == 0)) ||
        (!first && (int64_t)blockIdx.y * kApplyChunk >= n))
        return;
    const int32_t *row = p.table + (int64_t)b * p.max_blocks;
    const int2 *moves = p.moves + unit * p.max_moves;
    int err = 0;
    if (after > before || n < 0 || n > p.max_moves)
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
    if (first && layer == 0 && g == 0 && tid == 0 && p.seqlens != nullptr) {
        if (p.evicted != nullptr)
            p.evicted[b] += p.seqlens[b] - after;
        p.seqlens[b] = after;
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

constexpr int kPlanCached = 32768; // keys in shared memory at most; longer rows read theirs again

// Once per device: the plan kernel's shared memory.
bool plan_ready(int device)
{
    constexpr int kDevices = 64;
    static bool done[kDevices] = {};
    if (device < 0 || device >= kDevices)
        return false;
    if (!done[device])
        done[device] = cudaFuncSetAttribute(reinterpret_cast<const void *>(&evict_plan_kernel),
                                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            (kPlanCached + kEvictMaxSlots / 32) * 4) == cudaSuccess;
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
        num_moves == nullptr || row_lens == nullptr || !aligned16(mass) || !aligned16(slot_pos) || !aligned16(moves))
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
    p.cached = slots < kPlanCached ? slots : kPlanCached;
    const size_t smem = ((size_t)p.cached + (slots + 31) / 32) * sizeof(uint32_t);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !plan_ready(dev))
        return PKV_ECUDA;
    evict_plan_kernel<<<(unsigned)units, kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
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
    if (moves == nullptr || num_moves == nullptr || row_lens == nullptr || block_table == nullptr || !aligned16(moves) ||
        (cache_seqlens == nullptr && evicted != nullptr))
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
