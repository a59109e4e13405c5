// pkv_table.cu -- block tables that follow request lengths on the device: a
// page pool in device memory and one kernel that grows, shrinks and releases
// every row of a batch and lays out its new tokens ("flex_attention + paged
// KV + CUDA graphs vs vLLM", "What each option did": PageTable.reserve, here
// without the host).
//
// What is computed.  Row b holds held_b blocks and needs want_b = ceil((L_b +
// n_b) / P).  With take_b = max(0, want_b - held_b), give_b = max(0, held_b -
// want_b) and exclusive prefix sums T_b, R_b over the rows, block held_b + i of
// row b is ring[head + T_b + i], the page of its block want_b + i goes to
// ring[head + count + R_b + i], and token i of row b is token N_b + i of the
// ragged batch (N the prefix sum of n).  The pages handed out sit in
// [head, head + count) and those that come back go behind it, so the two
// never meet and every block and token can be done by any thread.
//
// How.  The prefix sums are over at most 1024 rows: every CTA does them again
// in shared memory (one row per thread, one scan for all three) instead of
// waiting for another, then the CTAs share out the warps' pieces of blocks and
// tokens.  The CTA that finishes last (a ticket in the pool's header; it never
// waits) writes what the others still read: held_blocks and the header.
//
// What bounds it.  A chain of dependent steps, not bytes: launch, the rows'
// numbers, the scan, a ring entry, a table entry or slot, held_blocks.  A step
// of 64 rows takes 4.9 us, of which the launch is 2; 1024 rows admitted at once,
// 3.75 MB, 8.8 us: 5.2 with neither pages nor lists (3.0 up to 256 rows: the scan
// over 32 warps for 8, and CTAs of 1024 threads), 2 for the slots and positions,
// 1.4 for the pages.  Measured on the way: a scan for every sum and test and 4096
// tokens a CTA 10.8 and 17.2 us; blocks and tokens in the same warps, one after
// the other, 6.8 and 9.6; a CTA per 2048, 1024, 512, 256 and 128 tokens 6.4,
// 5.9, 5.1, 4.9 and 4.9 for the step, no difference for the other.  1024 threads
// for a small batch cost 0.1 us, pieces of 32 tokens 0.2 at the large one.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kPoolHeader = 16; // int32 words before the ring
constexpr int kTableThreads = 1024;
constexpr int kTableMaxBatch = kTableThreads; // one row per thread
constexpr int kTablePiece = 64;               // tokens a warp lays out at a time
constexpr int kTableTokensPerCta = 256;
constexpr int kTableMaxPages = 1 << 30; // ring indices and their sums are 32-bit

struct TableParams {
    int32_t *pool;
    int32_t *table;
    int32_t *held;
    const int32_t *seqlens;
    const int32_t *new_tokens;
    int32_t *indptr;
    int64_t *slot_map;
    int32_t *positions;
    int32_t *err_flag;
    int cap; // pages of the ring: num_pages - 1
    int page_shift, max_blocks, batch, max_tokens;
};

// Inclusive prefix sums over the block's threads of K values at once; total
// gets the sums.
template <int K> __device__ __forceinline__ void block_scan(int64_t (&v)[K], int64_t (*s_warp)[32], int64_t (&total)[K])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v[k], o);
            if (lane >= o)
                v[k] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < K; ++k)
            s_warp[k][warp] = v[k];
    __syncthreads();
    // every warp adds the warps' sums up again, one per lane
#pragma unroll
    for (int k = 0; k < K; ++k) {
        int64_t x = lane < warps ? s_warp[k][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        total[k] = __shfl_sync(0xffffffffu, x, 31);
        const int64_t before = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
        v[k] += warp > 0 ? before : 0;
    }
    __syncthreads();
}

// The last row r in [lo, n) with first[r] <= t (first is non-decreasing).
__device__ __forceinline__ int row_of(const int *first, int lo, int n, int t)
{
    int hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kTableThreads) table_update_kernel(const TableParams p)
{
    __shared__ int64_t s_warp[3][32];
    __shared__ int s_take[kTableMaxBatch + 1], s_give[kTableMaxBatch + 1], s_tok[kTableMaxBatch + 1];
    __shared__ int s_len[kTableMaxBatch], s_held[kTableMaxBatch], s_want[kTableMaxBatch];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31;
    const int head = p.pool[0], count = p.pool[1];
    int err = 0;

    // 1. what row tid asks for
    int len = -1, held = 0;
    int64_t n = 0, want = 0;
    bool ok = false;
    if (tid < p.batch) {
        len = p.seqlens[tid];
        held = p.held[tid];
        n = len >= 0 && p.new_tokens != nullptr ? p.new_tokens[tid] : 0;
        const int64_t keys = len >= 0 ? len + n : 0;
        want = (keys + (1 << p.page_shift) - 1) >> p.page_shift;
        if (held < 0 || held > p.max_blocks)
            err = PKV_ERR_PAGE;
        else if (n < 0)
            err = PKV_ERR_QLEN;
        else if (want > p.max_blocks || keys > INT32_MAX)
            err = PKV_ERR_OVERFLOW;
        ok = err == 0;
        if (!ok)
            n = 0;
    }
    // 2. one prefix sum over the rows for tokens, pages taken and pages returned;
    // where the list or the pool is too short, again without the rows that fail
    const bool lists_tokens = p.slot_map != nullptr || p.positions != nullptr;
    int64_t take = 0, give = 0, sum[3], total[3];
    auto pages = [&] {
        take = ok && want > held ? want - held : 0;
        give = ok && held > want ? held - want : 0;
    };
    auto scan = [&] {
        sum[0] = n;
        sum[1] = take;
        sum[2] = give;
        block_scan<3>(sum, s_warp, total);
    };
    pages();
    scan();
    if (lists_tokens && total[0] > p.max_tokens) {
        if (n > 0 && sum[0] > p.max_tokens) {
            err |= PKV_ERR_QLEN;
            ok = false;
            n = 0;
        }
        pages();
        scan();
    }
    const bool pool_ok = head >= 0 && head < p.cap && count >= 0 && count <= p.cap && total[2] <= p.cap - count;
    if (!pool_ok || total[1] > count) { // the rows are served in order as long as the free pages last
        if (!pool_ok)
            err |= tid == 0 ? PKV_ERR_POOL : 0;
        else if (take > 0 && sum[1] > count)
            err |= PKV_ERR_POOL;
        if (!pool_ok || (take > 0 && sum[1] > count)) {
            ok = false;
            n = 0;
        }
        pages();
        scan();
    }
    const int64_t take_total = total[1], given_total = total[2];
    if (tid < p.batch) {
        s_len[tid] = len;
        s_held[tid] = held;
        s_want[tid] = ok ? (int)want : held;
        s_take[tid] = (int)(sum[1] - take);
        s_give[tid] = (int)(sum[2] - give);
        s_tok[tid] = (int)min(sum[0] - n, (int64_t)INT32_MAX);
        if (blockIdx.x == 0) {
            if (p.indptr != nullptr)
                p.indptr[tid] = s_tok[tid];
            set_error(p.err_flag, err);
        }
    }
    if (tid == 0) {
        s_take[p.batch] = (int)take_total;
        s_give[p.batch] = (int)given_total;
        s_tok[p.batch] = (int)min(total[0], (int64_t)INT32_MAX);
        if (blockIdx.x == 0 && p.indptr != nullptr)
            p.indptr[p.batch] = s_tok[p.batch];
    }
    __syncthreads();

    const int32_t *ring = p.pool + kPoolHeader;
    auto wrap = [&](int x) { return x >= p.cap ? x - p.cap : x; };
    // A page id out of the ring; 0 and a bit for one that cannot be.
    auto fresh = [&](int i) {
        const int id = ring[wrap(head + i)];
        if (id >= 1 && id <= p.cap)
            return id;
        err |= PKV_ERR_PAGE;
        return 0;
    };
    err = 0;
    const int step = (int)(gridDim.x * blockDim.x), first = (int)(blockIdx.x * blockDim.x) + tid;
    // 3. blocks taken, blocks returned.  Counted from the last warp and from the
    // middle one, so that a small call has blocks and tokens in different warps
    // and their loads under way at once.
    for (int64_t i = step - 1 - first; i < take_total; i += step) {
        const int b = row_of(s_take, 0, p.batch, (int)i);
        p.table[(int64_t)b * p.max_blocks + s_held[b] + ((int)i - s_take[b])] = fresh((int)i);
    }
    for (int64_t i = first < step / 2 ? first + step / 2 : first - step / 2; i < given_total; i += step) {
        const int b = row_of(s_give, 0, p.batch, (int)i);
        int32_t *entry = p.table + (int64_t)b * p.max_blocks + s_want[b] + ((int)i - s_give[b]);
        int id = *entry;
        if (id < 1 || id > p.cap) {
            err |= PKV_ERR_PAGE;
            id = 0;
        }
        *entry = 0;
        p.pool[kPoolHeader + wrap(wrap(head + count) + (int)i)] = id;
    }
    // 4. the new tokens' slots and positions: a warp's piece of consecutive tokens
    if (lists_tokens) {
        const int tokens = s_tok[p.batch];
        for (int64_t t0 = (int64_t)(first - lane) / 32 * kTablePiece; t0 < p.max_tokens;
             t0 += (int64_t)step / 32 * kTablePiece) {
            int b = 0;
            bool found = false;
#pragma unroll
            for (int k = 0; k < kTablePiece / 32; ++k) {
                const int64_t t = t0 + k * 32 + lane;
                if (t >= p.max_tokens)
                    break;
                int64_t slot = -1;
                int pos = -1;
                if (t < tokens) {
                    if (!found || s_tok[b + 1] <= t)
                        b = row_of(s_tok, b, p.batch, (int)t);
                    found = true;
                    pos = s_len[b] + ((int)t - s_tok[b]);
                    const int blk = pos >> p.page_shift;
                    const int id = blk < s_held[b] ? p.table[(int64_t)b * p.max_blocks + blk]
                                                   : fresh(s_take[b] + blk - s_held[b]);
                    if (id >= 1 && id <= p.cap)
                        slot = ((int64_t)id << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
                    else
                        err |= PKV_ERR_PAGE;
                }
                if (p.slot_map != nullptr)
                    p.slot_map[t] = slot;
                if (p.positions != nullptr)
                    p.positions[t] = pos;
            }
        }
    }
    set_error(p.err_flag, err);

    // 5. what every CTA has read by now
    __syncthreads();
    if (gridDim.x > 1) {
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(&p.pool[2], 1) == (int)gridDim.x - 1;
        }
        __syncthreads();
        if (!s_last)
            return;
    }
    if (tid < p.batch)
        p.held[tid] = s_want[tid];
    if (tid == 0) {
        p.pool[2] = 0;
        if (pool_ok) {
            p.pool[0] = wrap(head + (int)take_total);
            p.pool[1] = count - (int)take_total + (int)given_total;
        }
    }
}

__global__ void pool_init_kernel(int32_t *pool, int cap)
{
    const int i = (int)(blockIdx.x * blockDim.x) + (int)threadIdx.x;
    if (i < kPoolHeader)
        pool[i] = i == 1 ? cap : 0;
    if (i < cap)
        pool[kPoolHeader + i] = i + 1;
}

bool aligned4(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

} // namespace
} // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_device_pool_bytes(int32_t num_pages)
{
    return num_pages < 2 || num_pages > kTableMaxPages ? 0 : ((size_t)num_pages - 1 + kPoolHeader) * 4;
}

pkv_status pkv_device_pool_init(void *pool, size_t pool_bytes, int32_t num_pages, void *stream)
{
    if (pool == nullptr || num_pages < 2 || !aligned4(pool))
        return PKV_EINVAL;
    if (num_pages > kTableMaxPages)
        return PKV_EUNSUPPORTED;
    if (pool_bytes < pkv_device_pool_bytes(num_pages))
        return PKV_EINVAL;
    const int cap = num_pages - 1;
    pool_init_kernel<<<(cap > kPoolHeader ? cap - 1 : kPoolHeader - 1) / 256 + 1, 256, 0,
                       static_cast<cudaStream_t>(stream)>>>(static_cast<int32_t *>(pool), cap);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

pkv_status pkv_table_update(void *pool, int32_t num_pages, int32_t page_size, int32_t *block_table, int32_t max_blocks,
                            int32_t *held_blocks, const int32_t *cache_seqlens, const int32_t *new_tokens,
                            int32_t batch, int32_t *indptr, int64_t *slot_map, int32_t *positions, int32_t max_tokens,
                            int32_t *err_flag, void *stream)
{
    if (num_pages < 2 || page_size < 1 || max_blocks < 1 || batch < 0 || max_tokens < 0)
        return PKV_EINVAL;
    if (page_size > 256 || (page_size & (page_size - 1)) != 0 || batch > kTableMaxBatch ||
        num_pages > kTableMaxPages)
        return PKV_EUNSUPPORTED;
    if (batch == 0)
        return PKV_OK;
    if (pool == nullptr || block_table == nullptr || held_blocks == nullptr || cache_seqlens == nullptr)
        return PKV_EINVAL;
    if (!aligned4(pool) || !aligned4(block_table) || (reinterpret_cast<uintptr_t>(slot_map) & 7u) != 0)
        return PKV_EINVAL;
    TableParams p;
    p.pool = static_cast<int32_t *>(pool);
    p.table = block_table;
    p.held = held_blocks;
    p.seqlens = cache_seqlens;
    p.new_tokens = new_tokens;
    p.indptr = indptr;
    p.slot_map = slot_map;
    p.positions = positions;
    p.err_flag = err_flag;
    p.cap = num_pages - 1;
    p.page_shift = 0;
    while ((1 << p.page_shift) < page_size)
        ++p.page_shift;
    p.max_blocks = max_blocks;
    p.batch = batch;
    p.max_tokens = max_tokens;
    const int threads = batch <= 256 ? 256 : kTableThreads;
    int64_t grid = ((int64_t)max_tokens + kTableTokensPerCta - 1) / kTableTokensPerCta;
    const int64_t by_rows = (batch + 255) / 256; // each row may move many blocks without a token
    grid = grid < by_rows ? by_rows : grid;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return PKV_ECUDA;
    grid = grid > sm_count(dev) ? sm_count(dev) : grid;
    table_update_kernel<<<(unsigned)grid, threads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

} // extern "C"
