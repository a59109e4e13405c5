// pkv_tree.cu -- the whole-number side of speculative decoding with trees of
// drafted tokens: ancestor masks and positions, acceptance of the path the
// target model chose itself, and the move of the accepted tokens' K/V to the
// front of the row.  See include/pkv.h for the rules of each.
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kTreeNodes = 256;            // most nodes of a row
constexpr int kTreeWords = kTreeNodes / 32; // mask words of a node

// A row's node range; false (and a bit) where it is reversed or leaves the batch.
struct TreeRow {
    int first, nodes, len;
    bool ok;  // nodes are to be worked on
    int err;
};

__device__ __forceinline__ TreeRow tree_row(const int32_t *indptr, const int32_t *seqlens, int b, int total_q,
                                            int max_nodes)
{
    TreeRow r;
    r.first = indptr[b];
    const int64_t n = (int64_t)indptr[b + 1] - r.first;
    r.len = seqlens[b];
    r.err = 0;
    const bool listed = r.first >= 0 && n >= 0 && n <= (int64_t)total_q - r.first;
    r.nodes = listed ? (int)n : 0;
    if (!listed || n > max_nodes)
        r.err = PKV_ERR_QLEN;
    r.ok = r.err == 0 && r.len >= 0;
    return r;
}

// ---------------------------------------------------------------- masks

struct BuildParams {
    const int32_t *parents, *indptr, *seqlens;
    int32_t *mask, *positions, *err_flag;
    int total_q, max_nodes, words;
    bool whole; // mask rows in 16-byte pieces
};

// One CTA per row, one thread per node.  mask_i = bit i | mask_parent(i), by
// pointer doubling: each round ors in the mask of the node one hop up and
// doubles the hop, so a tree of depth d takes ceil(log2 d) rounds.  A node's
// ancestors come before it, so warps 0 .. 3 have nothing in words 4 .. 7; a node
// that has reached its root no longer reads or writes.  A row of s_mask is 12
// words: any 8 consecutive rows' 16-byte pieces lie in different banks.  Bound
// by shared memory (the masks of random parents) and by the chain of loads
// before it: 1024 rows of 129 .. 256 nodes, 7.9 MB, take 5.3 us (8.0 with the
// masks word by word and every node in every round; 6.1 with rows of 8 words
// written word by word, as other widths are), a few rows 2.0: the launch.
__global__ void __launch_bounds__(kTreeNodes) tree_build_kernel(const BuildParams p)
{
    __shared__ uint4 s_mask[kTreeNodes][3]; // (two are used)
    __shared__ int s_up[kTreeNodes];
    const TreeRow r = tree_row(p.indptr, p.seqlens, blockIdx.x, p.total_q, p.max_nodes);
    const int i = threadIdx.x;
    const bool mine = r.ok && i < r.nodes, high = i >= 128;
    int up = -1;
    if (mine)
        up = p.parents[r.first + i];
    const bool bad = __syncthreads_or(mine && (up < -1 || up >= i));
    if (i == 0)
        set_error(p.err_flag, r.err | (bad ? PKV_ERR_TREE : 0));
    const bool ok = r.ok && !bad;
    if (!ok) {
        const int64_t words = (int64_t)r.nodes * p.words;
        for (int64_t k = i; k < words; k += blockDim.x)
            p.mask[(int64_t)r.first * p.words + k] = 0;
        if (p.positions != nullptr)
            for (int64_t k = i; k < r.nodes; k += blockDim.x)
                p.positions[r.first + k] = -1;
        return;
    }
    const uint32_t bit = 1u << (i & 31);
    auto own = [&](int w) { return (i >> 5) == w ? bit : 0u; };
    uint4 lo = make_uint4(own(0), own(1), own(2), own(3)), hi = make_uint4(own(4), own(5), own(6), own(7));
    s_mask[i][0] = lo;
    s_mask[i][1] = hi;
    s_up[i] = up;
    while (__syncthreads_or(up >= 0)) {
        const bool more = up >= 0;
        if (more) {
            const uint4 x = s_mask[up][0];
            lo = make_uint4(lo.x | x.x, lo.y | x.y, lo.z | x.z, lo.w | x.w);
            if (high) {
                const uint4 y = s_mask[up][1];
                hi = make_uint4(hi.x | y.x, hi.y | y.y, hi.z | y.z, hi.w | y.w);
            }
            up = s_up[up];
        }
        __syncthreads();
        if (more) {
            s_mask[i][0] = lo;
            if (high)
                s_mask[i][1] = hi;
            s_up[i] = up;
        }
    }
    if (p.positions != nullptr && i < r.nodes)
        p.positions[r.first + i] = r.len - 1 + __popc(lo.x) + __popc(lo.y) + __popc(lo.z) + __popc(lo.w) +
                                   __popc(hi.x) + __popc(hi.y) + __popc(hi.z) + __popc(hi.w);
    if (p.whole) { // rows of 4 or 8 aligned words
        int32_t *out = p.mask + ((int64_t)r.first + i) * p.words;
        if (i < r.nodes) {
            *reinterpret_cast<uint4 *>(out) = lo;
            if (p.words == 8)
                *reinterpret_cast<uint4 *>(out + 4) = hi;
        }
        return;
    }
    // others: a warp's rows lie one after the other, consecutive lanes on consecutive words
    const int node0 = i & ~31, end = min(32, r.nodes - node0) * p.words;
    const uint32_t *rows = reinterpret_cast<const uint32_t *>(s_mask[node0]);
    for (int k = i & 31; k < end; k += 32)
        p.mask[((int64_t)r.first + node0) * p.words + k] = (int32_t)rows[k / p.words * 12 + k % p.words];
}

// ---------------------------------------------------------------- acceptance

struct AcceptParams {
    const int32_t *parents, *draft, *target, *root, *indptr, *seqlens;
    int32_t *path, *path_len, *next_token, *seqlens_out, *err_flag;
    int batch, total_q, max_nodes, max_path;
};

constexpr int kAcceptWarps = 4;

// One warp per row; each lane keeps the parents of nodes lane, lane + 32, ...
// and whether the node's drafted token is what the target chose at its parent.
// A step down the path is one ballot per 32 nodes.  Bound by the chain of four
// loads (range, parent, the parent's choice) and the ballots: 1024 rows of up to
// 129 nodes take 5.0 us, a few rows 2.8.
__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(const AcceptParams p)
{
    const int b = (int)blockIdx.x * kAcceptWarps + ((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= p.batch)
        return;
    const TreeRow r = tree_row(p.indptr, p.seqlens, b, p.total_q, p.max_nodes);
    const int root = p.root != nullptr ? p.root[b] : -1;
    int up[kTreeWords];
    bool bad = false;
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) {
        const int i = w * 32 + lane;
        up[w] = i; // no node's parent
        if (r.ok && i < r.nodes) {
            const int u = p.parents[r.first + i];
            bad |= u < -1 || u >= i;
            if (u >= -1 && u < i) {
                const bool fits = u < 0 ? p.root == nullptr || p.draft[r.first + i] == root
                                        : p.draft[r.first + i] == p.target[r.first + u];
                up[w] = fits ? u : i;
            }
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    int cur = -1, len = 0;
    if (r.ok && !bad) {
        while (len < p.max_path) {
            int next = -1;
#pragma unroll
            for (int w = 0; w < kTreeWords; ++w) {
                if (next < 0 && w * 32 < r.nodes) {
                    const uint32_t hit = __ballot_sync(0xffffffffu, up[w] == cur && w * 32 + lane > cur);
                    if (hit != 0)
                        next = w * 32 + __ffs(hit) - 1;
                }
            }
            if (next < 0)
                break;
            if (lane == 0)
                p.path[(int64_t)b * p.max_path + len] = next;
            cur = next;
            ++len;
        }
    }
    for (int k = len + lane; k < p.max_path; k += 32)
        p.path[(int64_t)b * p.max_path + k] = -1;
    if (lane == 0) {
        set_error(p.err_flag, r.err | (bad ? PKV_ERR_TREE : 0));
        p.path_len[b] = len;
        if (p.next_token != nullptr)
            p.next_token[b] = !r.ok || bad ? -1 : cur >= 0 ? p.target[r.first + cur] : root;
        if (p.seqlens_out != nullptr)
            p.seqlens_out[b] = r.len + len;
    }
}

// ---------------------------------------------------------------- commit

constexpr int kMaxLayers = 128;
constexpr int kCommitThreads = 256;
constexpr int kCommitAhead = 8; // tokens in flight per thread

struct CommitParams {
    void *k[kMaxLayers], *v[kMaxLayers];
    const int32_t *path, *path_len, *table, *seqlens;
    int32_t *err_flag;
    int max_path, max_blocks, page_shift, num_pages, num_kv_heads, head_dim, layout;
};

// One CTA per (row, layer).  The path rises (path[i] >= i), so a token's
// destination is never the source of a later one; each thread owns 16-byte
// pieces of a token's K or V, loads up to kCommitAhead tokens' pieces and then
// stores them, in path order.  The tokens that lie right already are the first
// ones (path[i] = i from some i on never again), and are skipped.  Bound by
// latency, the chain length, path, pages, data of every CTA: 36 layers x 64 rows
// of 8 heads of 128 are 2304 CTAs, a little over three waves, and take 15.1 us
// (75 MB read and written, with the tokens that stay), 5.9 of them when no token
// moves; HBM delivers 36 MB meanwhile, 38 % of its rate.  A small call takes 2.5.
// Measured: 4 tokens ahead 15.7 and 16 16.5 us; 128 threads 15.5, 512 20.2.
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const __grid_constant__ CommitParams p)
{
    __shared__ int64_t s_src[kTreeNodes], s_dst[kTreeNodes]; // elements, head 0
    __shared__ int s_stay; // first tokens that lie right
    const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
    const int L = p.seqlens[b], n = p.path_len[b];
    if (L < 0 || n == 0)
        return;
    int err = 0;
    if (n < 0 || n > p.max_path)
        err = PKV_ERR_TREE;
    if (tid == 0)
        s_stay = 0;
    __syncthreads();
    const int P = 1 << p.page_shift;
    const int32_t *path = p.path + (int64_t)b * p.max_path;
    const int32_t *row = p.table + (int64_t)b * p.max_blocks;
    auto element = [&](int page, int slot) {
        return p.layout == PKV_NHD ? (((int64_t)page << p.page_shift) + slot) * p.num_kv_heads * p.head_dim
                                   : ((int64_t)page * p.num_kv_heads * P + slot) * p.head_dim;
    };
    if (err == 0)
        for (int i = tid; i < n; i += kCommitThreads) {
            const int node = path[i];
            if (node < 0 || (i > 0 && node <= path[i - 1])) {
                err = PKV_ERR_TREE;
                continue;
            }
            const int64_t from = (int64_t)L + node, to = (int64_t)L + i;
            if (from >= (int64_t)p.max_blocks << p.page_shift || to >= (int64_t)p.max_blocks << p.page_shift) {
                err = PKV_ERR_OVERFLOW;
                continue;
            }
            const int page_from = row[from >> p.page_shift], page_to = row[to >> p.page_shift];
            if (page_from < 1 || page_from >= p.num_pages || page_to < 1 || page_to >= p.num_pages) {
                err = PKV_ERR_PAGE;
                continue;
            }
            if (node == i)
                atomicMax(&s_stay, i + 1);
            s_src[i] = element(page_from, (int)(from & (P - 1)));
            s_dst[i] = element(page_to, (int)(to & (P - 1)));
        }
    if (err != 0 && layer == 0)
        set_error(p.err_flag, err);
    if (__syncthreads_or(err))
        return;
    const int per_head = p.head_dim / 8, pieces = p.num_kv_heads * per_head;
    const int64_t head_step = p.layout == PKV_NHD ? p.head_dim : (int64_t)P * p.head_dim;
    for (int c = tid; c < 2 * pieces; c += kCommitThreads) {
        __nv_bfloat16 *pool = static_cast<__nv_bfloat16 *>(c < pieces ? p.k[layer] : p.v[layer]);
        const int x = c < pieces ? c : c - pieces;
        pool += x / per_head * head_step + x % per_head * 8;
        for (int i0 = s_stay; i0 < n; i0 += kCommitAhead) {
            uint4 piece[kCommitAhead];
#pragma unroll
            for (int k = 0; k < kCommitAhead; ++k)
                if (i0 + k < n)
                    piece[k] = *reinterpret_cast<const uint4 *>(pool + s_src[i0 + k]);
#pragma unroll
            for (int k = 0; k < kCommitAhead; ++k)
                if (i0 + k < n)
                    *reinterpret_cast<uint4 *>(pool + s_dst[i0 + k]) = piece[k];
        }
    }
}

bool sizes_ok(int32_t batch, int32_t total_q, int32_t max_nodes)
{
    return batch >= 0 && total_q >= 0 && max_nodes >= 1;
}

} // namespace
} // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_tree_build(const int32_t *parents, const int32_t *qo_indptr, const int32_t *cache_seqlens, int32_t batch,
                          int32_t total_q, int32_t max_nodes, int32_t *tree_mask, int32_t mask_words,
                          int32_t *positions, int32_t *err_flag, void *stream)
{
    if (!sizes_ok(batch, total_q, max_nodes) || mask_words < 1)
        return PKV_EINVAL;
    if (max_nodes > kTreeNodes || mask_words > kTreeWords)
        return PKV_EUNSUPPORTED;
    if (mask_words * 32 < max_nodes)
        return PKV_EINVAL;
    if (batch == 0 || total_q == 0)
        return PKV_OK;
    if (parents == nullptr || qo_indptr == nullptr || cache_seqlens == nullptr || tree_mask == nullptr)
        return PKV_EINVAL;
    BuildParams p;
    p.parents = parents;
    p.indptr = qo_indptr;
    p.seqlens = cache_seqlens;
    p.mask = tree_mask;
    p.positions = positions;
    p.err_flag = err_flag;
    p.total_q = total_q;
    p.max_nodes = max_nodes;
    p.words = mask_words;
    p.whole = mask_words % 4 == 0 && (reinterpret_cast<uintptr_t>(tree_mask) & 15u) == 0;
    const int threads = (max_nodes + 31) / 32 * 32;
    tree_build_kernel<<<batch, threads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

pkv_status pkv_tree_accept(const int32_t *parents, const int32_t *draft_tokens, const int32_t *target_tokens,
                           const int32_t *root_targets, const int32_t *qo_indptr, const int32_t *cache_seqlens,
                           int32_t batch, int32_t total_q, int32_t max_nodes, int32_t *path, int32_t max_path,
                           int32_t *path_len, int32_t *next_token, int32_t *seqlens_out, int32_t *err_flag,
                           void *stream)
{
    if (!sizes_ok(batch, total_q, max_nodes) || max_path < 1)
        return PKV_EINVAL;
    if (max_nodes > kTreeNodes)
        return PKV_EUNSUPPORTED;
    if (batch == 0)
        return PKV_OK;
    if (qo_indptr == nullptr || cache_seqlens == nullptr || path == nullptr || path_len == nullptr ||
        (total_q > 0 && (parents == nullptr || draft_tokens == nullptr || target_tokens == nullptr)))
        return PKV_EINVAL;
    AcceptParams p;
    p.parents = parents;
    p.draft = draft_tokens;
    p.target = target_tokens;
    p.root = root_targets;
    p.indptr = qo_indptr;
    p.seqlens = cache_seqlens;
    p.path = path;
    p.path_len = path_len;
    p.next_token = next_token;
    p.seqlens_out = seqlens_out;
    p.err_flag = err_flag;
    p.batch = batch;
    p.total_q = total_q;
    p.max_nodes = max_nodes;
    p.max_path = max_path;
    tree_accept_kernel<<<(batch + kAcceptWarps - 1) / kAcceptWarps, kAcceptWarps * 32, 0,
                         static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

pkv_status pkv_tree_commit(const pkv_cache_desc *desc, int32_t num_layers, void *const *k_caches,
                           void *const *v_caches, const int32_t *path, int32_t max_path, const int32_t *path_len,
                           const int32_t *block_table, int32_t max_blocks, const int32_t *cache_seqlens, int32_t batch,
                           int32_t *err_flag, void *stream)
{
    const pkv_status st = check_desc(desc);
    if (st != PKV_OK)
        return st;
    if (num_layers < 1 || max_path < 1 || max_blocks < 1 || batch < 0)
        return PKV_EINVAL;
    if (num_layers > kMaxLayers || max_path > kTreeNodes)
        return PKV_EUNSUPPORTED;
    if (k_caches == nullptr || v_caches == nullptr)
        return PKV_EINVAL;
    CommitParams p;
    for (int l = 0; l < num_layers; ++l) {
        p.k[l] = k_caches[l];
        p.v[l] = v_caches[l];
        if (p.k[l] == nullptr || p.v[l] == nullptr || ((reinterpret_cast<uintptr_t>(p.k[l]) |
                                                        reinterpret_cast<uintptr_t>(p.v[l])) & 15u) != 0)
            return PKV_EINVAL;
    }
    if (batch == 0)
        return PKV_OK;
    if (path == nullptr || path_len == nullptr || block_table == nullptr || cache_seqlens == nullptr)
        return PKV_EINVAL;
    p.path = path;
    p.path_len = path_len;
    p.table = block_table;
    p.seqlens = cache_seqlens;
    p.err_flag = err_flag;
    p.max_path = max_path;
    p.max_blocks = max_blocks;
    p.page_shift = 0;
    while ((1 << p.page_shift) < desc->page_size)
        ++p.page_shift;
    p.num_pages = desc->num_pages;
    p.num_kv_heads = desc->num_kv_heads;
    p.head_dim = desc->head_dim;
    p.layout = desc->layout;
    tree_commit_kernel<<<dim3(batch, num_layers), kCommitThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

} // extern "C"
