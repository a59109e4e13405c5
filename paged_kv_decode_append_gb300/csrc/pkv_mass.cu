// pkv_mass.cu -- attention weight that every cached token receives, added up
// over a step's queries and a kv head's query heads.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kMassThreads = 256;

struct MassParams {
    const __nv_bfloat16 *k_cache, *q;
    const int32_t *indptr, *table, *seqlens, *fresh_from, *evicted;
    const float *lse;
    float *mass;
    int32_t *pos, *err_flag;
    float scale;
    int batch, num_q_heads, num_kv_heads, group, head_dim, total_q, max_blocks, page_shift, num_pages, layout, slots;
};

// A warp per key, one row and kv head per CTA in x and y.
__global__ void __launch_bounds__(kMassThreads) mass_kernel(const __grid_constant__ MassParams p)
{
    const int b = blockIdx.x / p.num_kv_heads, g = blockIdx.x - b * p.num_kv_heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int L = p.seqlens[b];
    const int first = p.indptr != nullptr ? p.indptr[b] : b;
    const int64_t n = p.indptr != nullptr ? (int64_t)p.indptr[b + 1] - first : 1;
    int err = 0;
    if (first < 0 || n < 0 || n > (int64_t)p.total_q - first)
        err = PKV_ERR_QLEN;
    else if (L >= 0 && n > 0 &&
             L + n > min(min((int64_t)p.max_blocks << p.page_shift, (int64_t)p.slots), (int64_t)kMassMaxKeys))
        err = PKV_ERR_OVERFLOW;
    if (err != 0)
        set_error(p.err_flag, err);
    if (err != 0 || L < 0 || n == 0)
        return;
    const int keys = L + (int)n, D = p.head_dim;
    const int fresh = p.fresh_from != nullptr ? p.fresh_from[b] : L;
    const int64_t P = (int64_t)1 << p.page_shift;
    for (int t = blockIdx.y * (kMassThreads / 32) + warp; t < keys; t += gridDim.y * (kMassThreads / 32)) {
        const int64_t page = p.table[(int64_t)b * p.max_blocks + (t >> p.page_shift)], at = t & (P - 1);
        if (page < 1 || page >= p.num_pages) {
            set_error(p.err_flag, PKV_ERR_PAGE);
            continue;
        }
        const __nv_bfloat16 *k = p.k_cache + (p.layout == PKV_NHD ? ((page * P + at) * p.num_kv_heads + g) * D
                                                                 : ((page * p.num_kv_heads + g) * P + at) * D);
        float kv[8];
        for (int j = 0; j < D / 32; ++j)
            kv[j] = __bfloat162float(k[j * 32 + lane]);
        float sum = 0.f, part = 0.f;
        for (int i = max(0, t - L); i < n; ++i) {
            part = 0.f;
            for (int h = 0; h < p.group; ++h) {
                const int64_t head = ((int64_t)first + i) * p.num_q_heads + g * p.group + h;
                float s = 0.f;
                for (int j = 0; j < D / 32; ++j)
                    s += kv[j] * __bfloat162float(p.q[head * D + j * 32 + lane]);
                for (int d = 16; d > 0; d >>= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, d);
                const float z = p.lse[head];
                part += z == -INFINITY ? 0.f : expf(s * p.scale - z);
            }
            sum += part;
        }
        if (lane == 0) {
            const int64_t to = ((int64_t)b * p.num_kv_heads + g) * p.slots + t;
            p.mass[to] = t >= fresh ? sum : p.mass[to] + sum;
            if (t >= fresh && p.pos != nullptr)
                p.pos[to] = t + (p.evicted != nullptr ? p.evicted[b] : 0);
        }
    }
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
    if (batch > kMaxMassBatch || desc->page_size < 8 || s->group > 128 ||
        (int64_t)total_q * num_q_heads >= ((int64_t)1 << 31))
        return PKV_EUNSUPPORTED;
    s->bytes = 256;
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
        mass == nullptr || !aligned16(k_cache) || !aligned16(q) || !aligned16(lse) || !aligned16(mass) ||
        !aligned16(slot_pos))
        return PKV_EINVAL;
    if (workspace == nullptr || workspace_bytes < shape.bytes || !aligned16(workspace))
        return PKV_EWORKSPACE;
    MassParams p;
    p.k_cache = static_cast<const __nv_bfloat16 *>(k_cache);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.indptr = qo_indptr;
    p.table = block_table;
    p.seqlens = cache_seqlens;
    p.fresh_from = fresh_from;
    p.evicted = evicted;
    p.lse = lse;
    p.mass = mass;
    p.pos = slot_pos;
    p.err_flag = err_flag;
    p.scale = softmax_scale;
    p.batch = batch;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = desc->num_kv_heads;
    p.group = shape.group;
    p.head_dim = desc->head_dim;
    p.total_q = total_q;
    p.max_blocks = max_blocks;
    p.page_shift = 0;
    while ((1 << p.page_shift) < desc->page_size)
        ++p.page_shift;
    p.num_pages = desc->num_pages;
    p.layout = desc->layout;
    p.slots = slots;
    const int64_t keys = (int64_t)max_blocks * desc->page_size;
    const unsigned y = (unsigned)(keys / 8 + 1 < 512 ? keys / 8 + 1 : 512);
    mass_kernel<<<dim3((unsigned)batch * desc->num_kv_heads, y), kMassThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

} // extern "C"
