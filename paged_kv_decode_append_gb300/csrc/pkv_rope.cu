// pkv_rope.cu -- rotary positions of queries and new keys, and the append of
// the rotated keys to the paged cache in the same pass.
//
// What it computes.  Pair i of a head, (x, y), is turned by the angle 2 pi
// frac(pos F_i / 2^64) and scaled: (a (x cos - y sin), a (y cos + x sin)).  F_i
// is the pair's frequency in turns per token as a 64-bit fixed-point fraction,
// so that pos F_i modulo 2^64 is the fraction of a turn itself, exactly: a
// product of 32-bit floats would have lost the angle of position 10^6
// altogether.  (F_i as pkv_rope_freqs makes it, in 64-bit floats, is off by up to
// 2^-53 turns per token: 2^-33 of a turn at position 10^6.)  Its upper 32 bits
// are rounded to 24 for the sine, an angle off by at most 2^-25 of half a turn or
// 2^-23.3 radians; everything else is in 32 bits, rounded to bf16 once.
//
// What bounds it: memory.  Every q, k and v is read once and written once; the
// angles of a token are worked out once for all its heads.  16 prompts of 9,549
// tokens, 48 + 6 + 6 heads of 256 values (587 MB), take 91 us, 6.4 TB/s, 96 % of
// the copy rate.  A step of 2,044 tokens, 32 + 8 + 8 heads of 128 (50 MB), takes 9.2
// us with its data in L2, 16 us without; one token for each of 4 rows 3.1 us.
// With several tokens a CTA, which then share the look at the block table, those
// were 17 and 103 us: fewer loads are under way while the rows are looked up.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kRopeAhead = 4; // 32-byte items of a thread under way at once

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *q_out, *k_out;
    __nv_bfloat16 *k_cache, *v_cache; // NULL: no append
    const uint64_t *freqs;
    const int32_t *positions, *indptr, *evicted, *table, *seqlens;
    int32_t *err_flag;
    float attn_factor;
    int tokens, batch, num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved;
    int max_blocks, page_shift, num_pages, layout;
};

// What a CTA needs to know of one of its tokens.
struct RopeToken {
    int64_t slot; // element of (token's slot, head 0) in the pools; -1: not appended
    int64_t pos;
    int live;     // rotated at all
};

__device__ __forceinline__ bool rope_owns(const RopeParams &p, int b, int t)
{
    const int first = p.indptr[b], end = p.indptr[b + 1];
    return first >= 0 && first <= t && t < end && end <= p.tokens;
}

// Row of token t, or -1 (a whole warp).  Malformed ranges send the count of
// rows that begin at or before it astray; then every row is looked at, so that
// their neighbours are served.
__device__ __forceinline__ int rope_row(const RopeParams &p, int t, int lane)
{
    if (p.indptr == nullptr)
        return t;
    int n = 0;
    for (int b = 1 + lane; b < p.batch; b += 32) // (loads that do not wait for one another)
        n += p.indptr[b] <= t ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (rope_owns(p, n, t))
        return n;
    int found = p.batch;
    for (int b = lane; b < p.batch; b += 32)
        if (rope_owns(p, b, t)) {
            found = b;
            break;
        }
    found = __reduce_min_sync(0xffffffffu, found);
    return found < p.batch ? found : -1;
}

// Looks token t up (a whole warp).
__device__ __forceinline__ RopeToken rope_look_up(const RopeParams &p, int t, int lane)
{
    RopeToken tok = {-1, 0, 1};
    if (p.k_cache != nullptr) {
        const int b = rope_row(p, t, lane);
        const int L = b >= 0 ? p.seqlens[b] : -1;
        tok.live = L >= 0;
        if (L >= 0) {
            const int first = p.indptr == nullptr ? t : p.indptr[b];
            const int count = p.indptr == nullptr ? 1 : p.indptr[b + 1] - first;
            const int64_t at = (int64_t)L + (t - first);
            int bad = 0;
            tok.pos = at + (p.evicted != nullptr ? p.evicted[b] : 0);
            if ((int64_t)L + count > (int64_t)p.max_blocks << p.page_shift) {
                bad = PKV_ERR_OVERFLOW;
            } else { // a row is appended as a whole or not at all
                const int32_t *row = p.table + (int64_t)b * p.max_blocks;
                const int64_t page = row[at >> p.page_shift], in_page = at & ((1 << p.page_shift) - 1);
                const int end = (int)(((int64_t)L + count - 1) >> p.page_shift);
                for (int k = (L >> p.page_shift) + lane; k <= end; k += 32)
                    if (row[k] < 1 || row[k] >= p.num_pages)
                        bad = PKV_ERR_PAGE;
                bad = __any_sync(0xffffffffu, bad) ? PKV_ERR_PAGE : 0;
                if (bad == 0)
                    tok.slot = p.layout == PKV_NHD ? ((page << p.page_shift) + in_page) * p.num_kv_heads * p.head_dim
                                                   : ((page * p.num_kv_heads << p.page_shift) + in_page) * p.head_dim;
            }
            if (bad != 0 && lane == 0)
                set_error(p.err_flag, bad);
        }
    }
    if (p.positions != nullptr)
        tok.pos = p.positions[t];
    return tok;
}

// A CTA per token.  Its items of 32 bytes are 8 pairs of a head, or 16 values that
// are copied; a thread has the same place in the head in all of its items, and so
// the same angles.  kRopeAhead items at a time, and the next ones are read before
// those are turned and written: the first before the token's row is known, which
// one warp finds out meanwhile, with the angles.
template <int THREADS, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ RopeToken s_tok;
    __shared__ __align__(16) float s_cos[128], s_sin[128];
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const bool append = p.k_cache != nullptr;
    const int D = p.head_dim, half = p.rot_dim / 2;
    const int per_head = D / 16, heads_at_once = THREADS / per_head, j = tid % per_head;
    const int q_heads = p.q != nullptr ? p.num_q_heads : 0, k_heads = p.k != nullptr ? p.num_kv_heads : 0;
    const int heads = q_heads + k_heads + (append ? p.num_kv_heads : 0);
    const bool turns = 16 * j < p.rot_dim; // (heads of V do not)
    // the two 16-byte pieces of an item that turns, and of another
    const int e0 = turns && !INTERLEAVED ? 8 * j : 16 * j;
    const int e1 = turns && !INTERLEAVED ? half + 8 * j : 16 * j + 8;

    auto load = [&](int h0, uint4 (&a)[kRopeAhead], uint4 (&b)[kRopeAhead]) {
#pragma unroll
        for (int u = 0; u < kRopeAhead; ++u) {
            const int h = h0 + u * heads_at_once;
            if (h >= heads)
                continue;
            const bool is_v = h >= q_heads + k_heads;
            const __nv_bfloat16 *from = h < q_heads ? p.q + (t * q_heads + h) * D
                                        : is_v      ? p.v + (t * p.num_kv_heads + h - q_heads - k_heads) * D
                                                    : p.k + (t * p.num_kv_heads + h - q_heads) * D;
            a[u] = *reinterpret_cast<const uint4 *>(from + (is_v ? 16 * j : e0));
            b[u] = *reinterpret_cast<const uint4 *>(from + (is_v ? 16 * j + 8 : e1));
        }
    };
    int h0 = tid / per_head;
    uint4 a[kRopeAhead], b[kRopeAhead];
    load(h0, a, b);

    if (tid < 32) {
        const RopeToken tok = rope_look_up(p, (int)t, tid);
        for (int f = tid; f < half; f += 32) {
            const uint64_t turn = (uint64_t)tok.pos * p.freqs[f];
            float s, c; // 2^-31: half turns
            sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);
            s_cos[f] = c * p.attn_factor;
            s_sin[f] = s * p.attn_factor;
        }
        if (tid == 0)
            s_tok = tok;
    }
    __syncthreads();
    const RopeToken tok = s_tok;
    const int64_t head_step = p.layout == PKV_NHD ? D : (int64_t)D << p.page_shift;
    for (;;) {
#pragma unroll
        for (int u = 0; u < kRopeAhead; ++u) {
            const int h = h0 + u * heads_at_once;
            if (h >= heads)
                continue;
            const bool is_v = h >= q_heads + k_heads, pieces = turns && !is_v;
            const int g = h - q_heads - (is_v ? k_heads : 0);
            __nv_bfloat16 *to = nullptr, *also = nullptr;
            if (h < q_heads) {
                if (tok.live)
                    to = p.q_out + (t * q_heads + h) * D;
            } else {
                if (!is_v && p.k_out != nullptr)
                    also = p.k_out + (t * p.num_kv_heads + g) * D;
                if (tok.slot >= 0)
                    to = (is_v ? p.v_cache : p.k_cache) + tok.slot + g * head_step;
            }
            uint32_t w[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b[u].x, b[u].y, b[u].z, b[u].w};
            if (pieces) {
                const float4 *cp = reinterpret_cast<const float4 *>(s_cos) + 2 * j;
                const float4 *sp = reinterpret_cast<const float4 *>(s_sin) + 2 * j;
                const float4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
                const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (INTERLEAVED) {
#pragma unroll
                        for (int m = 0; m < 8; m += 4) { // words i and i + 4: pairs i and i + 4
                            const float2 y = bf16x2_to_float2(w[i + m]);
                            const __nv_bfloat162 r = __floats2bfloat162_rn(y.x * c[i + m] - y.y * s[i + m],
                                                                           y.y * c[i + m] + y.x * s[i + m]);
                            w[i + m] = *reinterpret_cast<const uint32_t *>(&r);
                        }
                    } else { // words i and i + 4: pairs 2 i and 2 i + 1
                        const float2 lo = bf16x2_to_float2(w[i]), hi = bf16x2_to_float2(w[i + 4]);
                        const __nv_bfloat162 r0 = __floats2bfloat162_rn(lo.x * c[2 * i] - hi.x * s[2 * i],
                                                                        lo.y * c[2 * i + 1] - hi.y * s[2 * i + 1]);
                        const __nv_bfloat162 r1 = __floats2bfloat162_rn(hi.x * c[2 * i] + lo.x * s[2 * i],
                                                                        hi.y * c[2 * i + 1] + lo.y * s[2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t *>(&r0);
                        w[i + 4] = *reinterpret_cast<const uint32_t *>(&r1);
                    }
                }
            }
            const uint4 y0 = make_uint4(w[0], w[1], w[2], w[3]), y1 = make_uint4(w[4], w[5], w[6], w[7]);
            const int o0 = is_v ? 16 * j : e0, o1 = is_v ? 16 * j + 8 : e1;
            if (to != nullptr) {
                *reinterpret_cast<uint4 *>(to + o0) = y0;
                *reinterpret_cast<uint4 *>(to + o1) = y1;
            }
            if (also != nullptr) {
                *reinterpret_cast<uint4 *>(also + o0) = y0;
                *reinterpret_cast<uint4 *>(also + o1) = y1;
            }
        }
        h0 += heads_at_once * kRopeAhead;
        if (h0 >= heads)
            break;
        load(h0, a, b);
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
    // 256 threads where a token has more items than 128 threads read at once
    const int heads = (p.q != nullptr ? p.num_q_heads : 0) + (p.k != nullptr ? p.num_kv_heads : 0) +
                      (p.k_cache != nullptr ? p.num_kv_heads : 0);
    if (heads * (p.head_dim / 16) <= 128 * kRopeAhead) {
        if (p.interleaved)
            rope_kernel<128, true><<<p.tokens, 128, 0, stream>>>(p);
        else
            rope_kernel<128, false><<<p.tokens, 128, 0, stream>>>(p);
    } else {
        if (p.interleaved)
            rope_kernel<256, true><<<p.tokens, 256, 0, stream>>>(p);
        else
            rope_kernel<256, false><<<p.tokens, 256, 0, stream>>>(p);
    }
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
        if (pair_of(low) <= 0.0) // not even pair 0 makes more than `low` turns
            first = -span;
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
    if (st != PKV_OK || num_tokens == 0) // (tensors of no tokens may have no address)
        return st;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (q == nullptr && k == nullptr))
        return PKV_EINVAL;
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
    if (batch < 0 || max_blocks < 1 || (append_indptr == nullptr && num_tokens != batch))
        return PKV_EINVAL;
    if (batch == 0 || num_tokens == 0)
        return PKV_OK;
    if ((q == nullptr) != (q_out == nullptr))
        return PKV_EINVAL;
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
