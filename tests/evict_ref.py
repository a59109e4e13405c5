"""Plain implementations of the rotary and eviction operators in 64 bits, row by
row, and the inputs their tests share."""
import math

import numpy as np
import torch

from paged_kv_decode_append_gb300 import workloads as wl


def rotate(x, pos, freqs, interleaved, factor=1.0):
    """x [T, heads, D] (float64) turned by 2 pi frac(pos f), f = freqs / 2^64 as
    whole numbers; returns the result and |x| + |y| of every value's pair."""
    R = 2 * len(freqs)
    turn = [[(int(p) * int(f)) % (1 << 64) for f in freqs] for p in pos]
    angle = np.array([[2 * math.pi * (t / 2.0 ** 64) for t in row] for row in turn]).reshape(len(pos), len(freqs))
    c, s = (factor * f(angle)[:, None] for f in (np.cos, np.sin))
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y, size = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = abs(factor) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def rotate_tol(y, size):
    """bf16 rounds by half a step, 2^-8 of the value.  Before that the angle is
    off by 2^-24 of half a turn through its 24 bits, 2^-22.3, sine and cosine by
    two steps of 2^-24 each, the factor's product, two products and a sum by
    2^-24 each: together below 2^-21 of |x| + |y|."""
    return 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * size


def row_keys(case, b, keys):
    """Row b's first `keys` keys, float64 [keys, Hkv, D]."""
    P = case.page_size
    pages = torch.as_tensor(case.block_table[b, : -(-keys // P)].astype(np.int64), device=case.k_cache.device)
    x = case.k_cache[pages]
    x = x if case.layout == wl.NHD else x.transpose(1, 2)
    return x.reshape(-1, case.num_kv_heads, case.head_dim)[:keys].double().cpu()


def lse_of(case, b, lo, n, L):
    """float64 log-sum-exps [n, Hq] of row b's n queries over its L + i + 1 keys."""
    k = row_keys(case, b, L + n)
    q = case.q[lo:lo + n].double().cpu()
    G = case.num_q_heads // case.num_kv_heads
    seen = torch.arange(L + n) <= L + torch.arange(n)[:, None]
    out = torch.empty(n, case.num_q_heads, dtype=torch.float64)
    for h in range(case.num_q_heads):
        a = (q[:, h] @ k[:, h // G].T * case.softmax_scale).masked_fill(~seen, -math.inf)
        out[:, h] = torch.logsumexp(a, 1)
    return out


def mass_row(case, b, lo, n, L, lse):
    """What row b's queries give to its keys, [Hkv, L + n] in 64 bits, and the
    bound of a correct kernel's error in it.

    The bound.  A weight is off by a relative delta: the score's products are
    exact in fp32 and summed over head_dim there (at most head_dim 2^-24 of scale
    sum |q k|, at most twice that through the base-2 scaling), the scaled score
    and lse are rounded on the way (2^-22 of each), exp2 is off by 2^-22.  Sums
    of positive fp32 terms: runs of at most 512 of them (2^-15 of the sum), their
    totals with no more than a few roundings."""
    k = row_keys(case, b, L + n)
    q = case.q[lo:lo + n].double().cpu()
    z = lse[lo:lo + n].double().cpu()
    G, D = case.num_q_heads // case.num_kv_heads, case.head_dim
    seen = torch.arange(L + n) <= L + torch.arange(n)[:, None]
    got = torch.zeros(case.num_kv_heads, L + n, dtype=torch.float64)
    tol = torch.zeros_like(got)
    for h in range(case.num_q_heads):
        s = q[:, h] @ k[:, h // G].T * case.softmax_scale
        size = q[:, h].abs() @ k[:, h // G].abs().T * abs(case.softmax_scale)
        w = torch.where(seen & (z[:, h] > -math.inf)[:, None], torch.exp(s - z[:, h][:, None]), 0.0)
        delta = 2 * D * 2.0 ** -24 * size + 2.0 ** -22 * (s.abs() + z[:, h].abs()[:, None] + 1)
        got[h // G] += w.sum(0)
        tol[h // G] += torch.where(w > 0, w * torch.expm1(delta), 0.0).sum(0)
    return got.numpy(), (tol + 2.0 ** -15 * got).numpy()


def plan_row(mass, pos, L, gone, budget, sink, recent):
    """(moves, kept slots in front) of one row of one head; None where it keeps all."""
    keep = L if budget < 0 else min(L, budget)
    if keep >= L:
        return []
    m = mass[:L].astype(np.float64)
    safe = (pos[:L] < sink) | (pos[:L].astype(np.int64) >= L + gone - recent)
    nan = np.isnan(m)
    order = sorted(range(L), key=lambda i: (not safe[i], nan[i], 0.0 if nan[i] else -m[i], i))
    stay = np.zeros(L, bool)
    stay[order[:keep]] = True
    src = [i for i in range(keep, L) if stay[i]]
    dst = [i for i in range(keep) if not stay[i]]
    return list(zip(src, dst))


def slot_rows(pool, layout, page_size, table_row, slots, head):
    """A kv head's rows at the given slots of one row: [slots, D], and a setter."""
    page = torch.as_tensor(table_row[np.asarray(slots) // page_size].astype(np.int64), device=pool.device)
    at = torch.as_tensor(np.asarray(slots) % page_size, device=pool.device)
    view = pool if layout == wl.NHD else pool.transpose(1, 2)
    return view, page, at, head


def move_slots(pool, layout, page_size, table_row, moves, head):
    """The moves of one row and head in one pool."""
    if not moves:
        return
    src, dst = zip(*moves)
    view, page, at, _ = slot_rows(pool, layout, page_size, table_row, src, head)
    rows = view[page, at, head].clone()
    view, page, at, _ = slot_rows(pool, layout, page_size, table_row, dst, head)
    view[page, at, head] = rows
