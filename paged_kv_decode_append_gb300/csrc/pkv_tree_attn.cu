// pkv_tree_attn.cu -- attention of a tree of drafted tokens over the paged
// cache: node i of row b attends the row's L_b cached keys and drafted key j
// iff bit j of its mask is set (include/pkv.h).
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

struct TreeParams {
    const __nv_bfloat16 *q, *k, *v;
    const int32_t *indptr, *mask, *table, *seqlens;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *err_flag;
    int batch, num_q_heads, num_kv_heads, total_q, max_blocks, max_nodes, words;
    int page_shift, num_pages, layout;
    float q_scale;
};

constexpr int kTreeWarps = 4;
constexpr float kLn2 = 0.693147180559945309f;

// One CTA per (node, query head), its warps on every kTreeWarps-th key: dot
// product over the lanes, online softmax per warp, merged in shared memory.
template <int D>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_attn_kernel(const TreeParams p)
{
    constexpr int kPer = D / 32;
    __shared__ float s_m[kTreeWarps], s_l[kTreeWarps], s_o[kTreeWarps][D];
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = 0, hi = p.batch - 1; // last row whose range starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.indptr[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int b = lo, first = p.indptr[b];
    const int64_t n = (int64_t)p.indptr[b + 1] - first;
    if (first < 0 || n < 0 || n > (int64_t)p.total_q - first) {
        if (threadIdx.x == 0)
            set_error(p.err_flag, PKV_ERR_QLEN);
        return;
    }
    if (t < first || t >= first + n)
        return;
    const int L = p.seqlens[b];
    const int64_t keys = (int64_t)L + n;
    const int32_t *row = p.table + (int64_t)b * p.max_blocks;
    int err = 0;
    bool zero = L < 0;
    if (!zero && n > p.max_nodes)
        err = PKV_ERR_QLEN;
    else if (!zero && keys > ((int64_t)p.max_blocks << p.page_shift))
        err = PKV_ERR_OVERFLOW;
    else if (!zero) {
        int bad = 0;
        for (int64_t k = threadIdx.x; (k << p.page_shift) < keys; k += kTreeWarps * 32)
            bad |= row[k] < 1 || row[k] >= p.num_pages;
        if (__syncthreads_or(bad))
            err = PKV_ERR_PAGE;
    }
    if (n > p.max_nodes)
        err = PKV_ERR_QLEN;
    if (threadIdx.x == 0)
        set_error(p.err_flag, err);
    zero |= err != 0;
    const int g = h / (p.num_q_heads / p.num_kv_heads);
    const __nv_bfloat16 *q = p.q + ((int64_t)t * p.num_q_heads + h) * D;
    float x[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        x[e] = __bfloat162float(q[e * 32 + lane]) * p.q_scale;
        o[e] = 0.f;
    }
    for (int64_t k = warp; !zero && k < keys; k += kTreeWarps) {
        const int j = (int)(k - L);
        if (j >= 0 && !((uint32_t)p.mask[(int64_t)t * p.words + (j >> 5)] >> (j & 31) & 1u))
            continue;
        const int64_t page = row[k >> p.page_shift], slot = k & ((1 << p.page_shift) - 1);
        const int64_t at = p.layout == PKV_NHD ? (((page << p.page_shift) + slot) * p.num_kv_heads + g) * D
                                               : (((page * p.num_kv_heads + g) << p.page_shift) + slot) * D;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            s += x[e] * __bfloat162float(p.k[at + e * 32 + lane]);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, w);
        const float top = fmaxf(m, s), scale = exp2f(m - top), e2 = exp2f(s - top);
        m = top;
        l = l * scale + e2;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            o[e] = o[e] * scale + e2 * __bfloat162float(p.v[at + e * 32 + lane]);
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        s_o[warp][e * 32 + lane] = o[e];
    __syncthreads();
    float top = -INFINITY, total = 0.f;
    for (int w = 0; w < kTreeWarps; ++w)
        top = fmaxf(top, s_m[w]);
    for (int w = 0; w < kTreeWarps; ++w)
        total += s_m[w] == -INFINITY ? 0.f : s_l[w] * exp2f(s_m[w] - top);
    for (int c = threadIdx.x; c < D; c += kTreeWarps * 32) {
        float sum = 0.f;
        for (int w = 0; w < kTreeWarps; ++w)
            sum += s_m[w] == -INFINITY ? 0.f : s_o[w][c] * exp2f(s_m[w] - top);
        p.out[((int64_t)t * p.num_q_heads + h) * D + c] = __float2bfloat16_rn(total == 0.f ? 0.f : sum / total);
    }
    if (threadIdx.x == 0 && p.lse != nullptr)
        p.lse[(int64_t)t * p.num_q_heads + h] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
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
    if (batch > kMaxTreeBatch || max_nodes > kTreeMaxNodes || desc->page_size < 8 || s->group > 128 ||
        (int64_t)total_q * num_q_heads >= ((int64_t)1 << 31))
        return PKV_EUNSUPPORTED;
    s->bytes = 256;
    return PKV_OK;
}

cudaError_t launch_tree_attn(const TreeArgs &a, cudaStream_t stream)
{
    TreeParams p;
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k = static_cast<const __nv_bfloat16 *>(a.k_cache);
    p.v = static_cast<const __nv_bfloat16 *>(a.v_cache);
    p.indptr = a.qo_indptr;
    p.mask = a.tree_mask;
    p.table = a.block_table;
    p.seqlens = a.cache_seqlens;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.lse = a.lse;
    p.err_flag = a.err_flag;
    p.batch = a.batch;
    p.num_q_heads = a.num_q_heads;
    p.num_kv_heads = a.desc.num_kv_heads;
    p.total_q = a.total_q;
    p.max_blocks = a.max_blocks;
    p.max_nodes = a.max_nodes;
    p.words = a.mask_words;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.desc.page_size)
        ++p.page_shift;
    p.num_pages = a.desc.num_pages;
    p.layout = a.desc.layout;
    p.q_scale = a.q_scale;
    const dim3 grid(a.total_q, a.num_q_heads);
    if (a.desc.head_dim == 64)
        tree_attn_kernel<64><<<grid, kTreeWarps * 32, 0, stream>>>(p);
    else if (a.desc.head_dim == 128)
        tree_attn_kernel<128><<<grid, kTreeWarps * 32, 0, stream>>>(p);
    else
        tree_attn_kernel<256><<<grid, kTreeWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace pkv
