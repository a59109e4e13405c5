// pkv_rope.cu -- rotary positions of queries and new keys, and the append of
// the rotated keys to the paged cache in the same pass.
//
// What it computes.  Pair i of a head, (x, y), is turned by the angle 2 pi
// frac(pos F_i / 2^64) and scaled: (a (x cos - y sin), a (y cos + x sin)).  F_i
// is the pair's frequency in turns per token as a 64-bit fixed-point fraction,
// so that pos F_i modulo 2^64 is the fraction of a turn itself, exact but for
// the rounding of F_i (2^-65 pos turns): a product of 32-bit floats would have
// lost the angle of position 10^6 altogether.  Its upper 32 bits are rounded
// to 24 for the sine (an angle off by at most 2^-24); everything else is in 32
// bits, rounded to bf16 once.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 8; // tokens of a CTA at most: one warp looks each up
constexpr int kRopeAhead = 4;  // 32-byte items of a thread under way at once

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out;
    __nv_bfloat16 *k_cache, *v_cache; // NULL: no append
    const uint64_t *freqs;
    const int32_t *positions, *indptr, *evicted, *table, *seqlens;
    int32_t *err_flag;
    float attn_factor;
    int tokens, per_cta, batch, num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved;
    int max_blocks, page_shift, num_pages, layout;
};

// What a CTA needs to know of one of its tokens.
struct RopeToken {
    int64_t slot; // element of (token's slot, head 0) in the pools; -1: not appended
    int64_t pos;
    int row, live; // live: rotated at all
};

__device__ __forceinline__ bool rope_owns(const RopeParams &p, int b, int t)
{
    const int first = p.indptr[b], end = p.indptr[b + 1];
    return first >= 0 && first <= t && t < end && end <= p.tokens;
}

// Row of token t, or -1 (a whole warp).  Malformed ranges send the bisection
// astray; then every row is looked at, so that their neighbours are served.
__device__ __forceinline__ int rope_row(const RopeParams &p, int t, int lane)
{
    if (p.indptr == nullptr)
        return t;
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.indptr[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    if (rope_owns(p, lo, t))
        return lo;
    int found = p.batch;
    for (int b = lane; b < p.batch; b += 32)
        if (rope_owns(p, b, t)) {
            found = b;
            break;
        }
    found = __reduce_min_sync(0xffffffffu, found);
    return found < p.batch ? found : -1;
}

__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ RopeToken s_tok[kRopeTokens];
    __shared__ int s_bad[kRopeTokens]; // of the row that first appears at this token: its error
    extern __shared__ float s_cs[];    // [token][cos | sin][rot_dim / 2]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * p.per_cta, n = min(p.per_cta, p.tokens - t0);
    const bool append = p.k_cache != nullptr;
    const int D = p.head_dim, half = p.rot_dim / 2;

    if (warp < n) { // a warp for each token
        const int t = t0 + warp;
        RopeToken tok = {-1, 0, -1, 1};
        int bad = 0;
        if (append) {
            const int b = rope_row(p, t, lane);
            const int L = b >= 0 ? p.seqlens[b] : -1;
            tok.row = b;
            tok.live = L >= 0;
            if (L >= 0) {
                const int first = p.indptr == nullptr ? t : p.indptr[b];
                const int count = p.indptr == nullptr ? 1 : p.indptr[b + 1] - first;
                const int64_t at = (int64_t)L + (t - first);
                tok.pos = at + (p.evicted != nullptr ? p.evicted[b] : 0);
                // a row is appended as a whole or not at all; its first token in this CTA looks
                if ((int64_t)L + count > (int64_t)p.max_blocks << p.page_shift) {
                    bad = PKV_ERR_OVERFLOW;
                } else {
                    const int32_t *row = p.table + (int64_t)b * p.max_blocks;
                    if (warp == 0 || t == first) {
                        const int last = (int)(((int64_t)L + count - 1) >> p.page_shift);
                        for (int k = (L >> p.page_shift) + lane; k <= last; k += 32)
                            if (row[k] < 1 || row[k] >= p.num_pages)
                                bad = PKV_ERR_PAGE;
                        bad = __any_sync(0xffffffffu, bad) ? PKV_ERR_PAGE : 0;
                    }
                    const int64_t page = row[at >> p.page_shift], in_page = at & ((1 << p.page_shift) - 1);
                    if (page < 1 || page >= p.num_pages)
                        bad = PKV_ERR_PAGE;
                    else
                        tok.slot = p.layout == PKV_NHD
                                       ? ((page << p.page_shift) + in_page) * p.num_kv_heads * D
                                       : ((page * p.num_kv_heads << p.page_shift) + in_page) * D;
                }
            }
        }
        if (p.positions != nullptr)
            tok.pos = p.positions[t];
        if (lane == 0) {
            s_tok[warp] = tok;
            s_bad[warp] = bad;
            if (bad != 0)
                set_error(p.err_flag, bad);
        }
    }
    __syncthreads();
    for (int i = tid; i < n * half; i += kRopeThreads) {
        const int k = i / half, f = i - k * half;
        const uint64_t turn = (uint64_t)s_tok[k].pos * p.freqs[f];
        float s, c; // 2^-31: half turns
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);
        s_cs[2 * k * half + f] = c * p.attn_factor;
        s_cs[(2 * k + 1) * half + f] = s * p.attn_factor;
    }
    __syncthreads();

    // Items of 32 bytes: 8 pairs of a head, or 16 values that are copied.  A
    // thread has the same place in the head in all of its items.
    const int per_head = D / 16, heads_at_once = kRopeThreads / per_head;
    const int j = tid % per_head;
    const int q_heads = p.q != nullptr ? p.num_q_heads : 0, k_heads = p.k != nullptr ? p.num_kv_heads : 0;
    const int heads = q_heads + k_heads + (append ? p.num_kv_heads : 0);
    const int items = n * heads;
    const int64_t head_step = p.layout == PKV_NHD ? D : (int64_t)D << p.page_shift;
    const bool rotated = 16 * j < p.rot_dim;
    // the two 16-byte pieces of an item
    const int e0 = rotated && !p.interleaved ? 8 * j : 16 * j;
    const int e1 = rotated && !p.interleaved ? half + 8 * j : 16 * j + 8;
    for (int x0 = tid / per_head; x0 < items; x0 += heads_at_once * kRopeAhead) {
        uint4 a[kRopeAhead], b[kRopeAhead];
        __nv_bfloat16 *to[kRopeAhead], *also[kRopeAhead];
        int cs[kRopeAhead]; // token, or -1 for a copy
#pragma unroll
        for (int u = 0; u < kRopeAhead; ++u) {
            const int x = x0 + u * heads_at_once;
            to[u] = also[u] = nullptr;
            if (x >= items)
                continue;
            const int k = x / heads, h = x - k * heads;
            const RopeToken &tok = s_tok[k];
            const int64_t t = t0 + k;
            if (!tok.live)
                continue;
            const __nv_bfloat16 *from;
            if (h < q_heads) {
                const int64_t at = (t * q_heads + h) * D;
                from = p.q + at;
                to[u] = p.q_out + at;
                cs[u] = rotated ? k : -1;
            } else {
                const bool is_k = h < q_heads + k_heads;
                const int g = is_k ? h - q_heads : h - q_heads - k_heads;
                const int64_t at = (t * p.num_kv_heads + g) * D;
                from = (is_k ? p.k : p.v) + at;
                cs[u] = is_k && rotated ? k : -1;
                if (is_k && p.k_out != nullptr)
                    also[u] = p.k_out + at;
                if (append && tok.slot >= 0) {
                    int first = k; // the token that looked at the row's pages
                    while (first > 0 && s_tok[first - 1].row == tok.row)
                        --first;
                    if (s_bad[first] == 0)
                        to[u] = (is_k ? p.k_cache : p.v_cache) + tok.slot + g * head_step;
                }
                if (to[u] == nullptr && also[u] == nullptr)
                    continue;
            }
            const bool pieces = cs[u] >= 0;
            a[u] = *reinterpret_cast<const uint4 *>(from + (pieces ? e0 : 16 * j));
            b[u] = *reinterpret_cast<const uint4 *>(from + (pieces ? e1 : 16 * j + 8));
        }
#pragma unroll
        for (int u = 0; u < kRopeAhead; ++u) {
            if (to[u] == nullptr && also[u] == nullptr)
                continue;
            const bool pieces = cs[u] >= 0;
            if (pieces) {
                const float4 *cp = reinterpret_cast<const float4 *>(s_cs + 2 * cs[u] * half + 8 * j);
                const float4 *sp = reinterpret_cast<const float4 *>(s_cs + (2 * cs[u] + 1) * half + 8 * j);
                const float4 c4[2] = {cp[0], cp[1]}, s4[2] = {sp[0], sp[1]};
                const float *c = &c4[0].x, *s = &s4[0].x;
                uint32_t w[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (p.interleaved) {
#pragma unroll
                        for (int m = 0; m < 2; ++m) { // words i and i + 4: pairs i and i + 4
                            const float2 z = bf16x2_to_float2(w[i + 4 * m]);
                            const float cc = c[i + 4 * m], ss = s[i + 4 * m];
                            const __nv_bfloat162 r = __floats2bfloat162_rn(z.x * cc - z.y * ss, z.y * cc + z.x * ss);
                            w[i + 4 * m] = *reinterpret_cast<const uint32_t *>(&r);
                        }
                    } else { // words i and i + 4: pairs 2 i and 2 i + 1
                        const float2 lo = bf16x2_to_float2(w[i]), hi = bf16x2_to_float2(w[i + 4]);
                        const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
                        const __nv_bfloat162 r0 = __floats2bfloat162_rn(lo.x * c0 - hi.x * s0, lo.y * c1 - hi.y * s1);
                        const __nv_bfloat162 r1 = __floats2bfloat162_rn(hi.x * c0 + lo.x * s0, hi.y * c1 + lo.y * s1);
                        w[i] = *reinterpret_cast<const uint32_t *>(&r0);
                        w[i + 4] = *reinterpret_cast<const uint32_t *>(&r1);
                    }
                }
                a[u] = make_uint4(w[0], w[1], w[2], w[3]);
                b[u] = make_uint4(w[4], w[5], w[6], w[7]);
            }
            const int o0 = pieces ? e0 : 16 * j, o1 = pieces ? e1 : 16 * j + 8;
            if (to[u] != nullptr) {
                *reinterpret_cast<uint4 *>(to[u] + o0) = a[u];
                *reinterpret_cast<uint4 *>(to[u] + o1) = b[u];
            }
            if (also[u] != nullptr) {
                *reinterpret_cast<uint4 *>(also[u] + o0) = a[u];
                *reinterpret_cast<uint4 *>(also[u] + o1) = b[u];
            }
        }
    }
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// What pkv_rope and pkv_rope_append check alike.
pkv_status rope_check(int head_dim, int num_q_heads, int num_kv_heads, int num_tokens, int rot_dim, int pairing,
                      float attn_factor)
{
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || rot_dim < 1 || rot_dim > head_dim ||
        (pairing != PKV_ROPE_HALF && pairing != PKV_ROPE_INTERLEAVED) || !isfinite(attn_factor))
        return PKV_EINVAL;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || rot_dim % 16 != 0)
        return PKV_EUNSUPPORTED;
    return PKV_OK;
}

pkv_status launch_rope(RopeParams &p, cudaStream_t stream)
{
    // tokens of a CTA: more share a look at the page table, as long as every SM has CTAs enough
    p.per_cta = p.tokens <= 1216 ? 1 : p.tokens <= 4864 ? 4 : kRopeTokens;
    const size_t smem = (size_t)p.per_cta * p.rot_dim * sizeof(float);
    rope_kernel<<<(p.tokens + p.per_cta - 1) / p.per_cta, kRopeThreads, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

} // namespace
} // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor, double low, double high,
                          double orig_len, uint64_t *freqs, float *attn_factor)
{
    constexpr double kTurn = 6.283185307179586476925286766559;
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !isfinite(base) || freqs == nullptr)
        return PKV_EINVAL;
    const bool stretched = scaling != PKV_ROPE_PLAIN;
    if (scaling < PKV_ROPE_PLAIN || scaling > PKV_ROPE_TURNS)
        return PKV_EINVAL;
    if (stretched && (!(factor >= 1.0) || !isfinite(factor)))
        return PKV_EINVAL;
    if (scaling == PKV_ROPE_NTK && rot_dim < 4)
        return PKV_EINVAL;
    if ((scaling == PKV_ROPE_PARTS || scaling == PKV_ROPE_TURNS) &&
        (!(low > 0.0) || !(high > low) || !isfinite(high) || !(orig_len > 0.0) || !isfinite(orig_len)))
        return PKV_EINVAL;
    const double R = rot_dim;
    if (scaling == PKV_ROPE_NTK)
        base *= pow(factor, R / (R - 2.0));
    // pair that makes `turns` turns over orig_len tokens
    auto pair_of = [&](double turns) { return R * log(orig_len / (kTurn * turns)) / (2.0 * log(base)); };
    double first = 0.0, span = 1.0;
    if (scaling == PKV_ROPE_PARTS) {
        first = fmax(floor(pair_of(high)), 0.0);
        span = fmax(fmin(ceil(pair_of(low)), R - 1.0) - first, 1e-3);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / R);
        double part = 0.0; // of f that is stretched
        if (scaling == PKV_ROPE_LINEAR)
            part = 1.0;
        else if (scaling == PKV_ROPE_PARTS)
            part = fmin(fmax((i - first) / span, 0.0), 1.0);
        else if (scaling == PKV_ROPE_TURNS)
            part = 1.0 - fmin(fmax((orig_len * f / kTurn - low) / (high - low), 0.0), 1.0);
        f = f / factor * part + f * (1.0 - part);
        // turns per token, below 1/6: 2^-64 of a turn fits in 64 bits
        freqs[i] = (uint64_t)(ldexp(f / kTurn, 64) + 0.5);
    }
    if (attn_factor != nullptr)
        *attn_factor = scaling == PKV_ROPE_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return PKV_OK;
}

pkv_status pkv_rope(const void *q, const void *k, const int32_t *positions, int32_t num_tokens, int32_t num_q_heads,
                    int32_t num_kv_heads, int32_t head_dim, const uint64_t *freqs, int32_t rot_dim, int32_t pairing,
                    float attn_factor, void *q_out, void *k_out, void *stream)
{
    const pkv_status st = rope_check(head_dim, num_q_heads, num_kv_heads, num_tokens, rot_dim, pairing, attn_factor);
    if (st != PKV_OK)
        return st;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (q == nullptr && k == nullptr))
        return PKV_EINVAL;
    if (num_tokens == 0)
        return PKV_OK;
    if (freqs == nullptr || positions == nullptr || (q != nullptr && num_q_heads < 1) ||
        (k != nullptr && num_kv_heads < 1) || !aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
        return PKV_EINVAL;
    RopeParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.freqs = freqs;
    p.positions = positions;
    p.attn_factor = attn_factor;
    p.tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rot_dim = rot_dim;
    p.interleaved = pairing == PKV_ROPE_INTERLEAVED;
    return launch_rope(p, static_cast<cudaStream_t>(stream));
}

pkv_status pkv_rope_append(const pkv_cache_desc *desc, void *k_cache, void *v_cache, const void *q, const void *k_new,
                           const void *v_new, int32_t num_tokens, const int32_t *append_indptr,
                           const int32_t *positions, const int32_t *evicted, const uint64_t *freqs, int32_t rot_dim,
                           int32_t pairing, float attn_factor, const int32_t *block_table, int32_t max_blocks,
                           const int32_t *cache_seqlens, int32_t batch, int32_t num_q_heads, void *q_out,
                           int32_t *err_flag, void *stream)
{
    pkv_status st = check_desc(desc);
    if (st == PKV_OK)
        st = rope_check(desc->head_dim, num_q_heads, desc->num_kv_heads, num_tokens, rot_dim, pairing, attn_factor);
    if (st != PKV_OK)
        return st;
    if (batch < 0 || max_blocks < 1 || (q == nullptr) != (q_out == nullptr) ||
        (append_indptr == nullptr && num_tokens != batch))
        return PKV_EINVAL;
    if (batch == 0 || num_tokens == 0)
        return PKV_OK;
    if (k_cache == nullptr || v_cache == nullptr || k_new == nullptr || v_new == nullptr || freqs == nullptr ||
        block_table == nullptr || cache_seqlens == nullptr || (q != nullptr && num_q_heads < 1))
        return PKV_EINVAL;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q) || !aligned16(k_new) || !aligned16(v_new) ||
        !aligned16(q_out))
        return PKV_EINVAL;
    RopeParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k_new);
    p.v = static_cast<const __nv_bfloat16 *>(v_new);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_cache = static_cast<__nv_bfloat16 *>(k_cache);
    p.v_cache = static_cast<__nv_bfloat16 *>(v_cache);
    p.freqs = freqs;
    p.positions = positions;
    p.indptr = append_indptr;
    p.evicted = evicted;
    p.table = block_table;
    p.seqlens = cache_seqlens;
    p.err_flag = err_flag;
    p.attn_factor = attn_factor;
    p.tokens = num_tokens;
    p.batch = batch;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = desc->num_kv_heads;
    p.head_dim = desc->head_dim;
    p.rot_dim = rot_dim;
    p.interleaved = pairing == PKV_ROPE_INTERLEAVED;
    p.max_blocks = max_blocks;
    while ((1 << p.page_shift) < desc->page_size)
        ++p.page_shift;
    p.num_pages = desc->num_pages;
    p.layout = desc->layout;
    return launch_rope(p, static_cast<cudaStream_t>(stream));
}

} // extern "C"
