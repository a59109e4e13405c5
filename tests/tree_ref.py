"""Plain implementations of the tree and table operators, row by row on the
host (the attention in 64 bits), and the inputs their tests share."""
import math

import numpy as np
import torch

from paged_kv_decode_append_gb300 import workloads as wl


def random_parents(rng, counts):
    """Random recursive trees: any earlier node, or -1 (the cache)."""
    return [rng.integers(-1, np.maximum(np.arange(n), 0)) if n else np.zeros(0, np.int64) for n in counts]


def ancestor_bits(parents):
    """Bool [n, n]: node i sees itself and its ancestors."""
    n = len(parents)
    seen = np.eye(n, dtype=bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] |= seen[p]
    return seen


def pack(rows, words):
    """Bool [n, n] per row -> int32 [sum n, words]."""
    out = []
    for seen in rows:
        n = len(seen)
        wide = np.zeros((n, words * 32), bool)
        wide[:, :n] = seen
        out.append(np.packbits(wide, axis=1, bitorder="little").view(np.int32).reshape(n, words))
    return np.concatenate(out) if out else np.zeros((0, words), np.int32)


def row_kv(case, b, n, with_new):
    """Row b's K and V over its cached and drafted tokens, float64 [keys, Hkv, D]."""
    L, P = int(case.cache_seqlens[b]), case.page_size
    lo = int(case.qo_indptr[b])
    pages = torch.as_tensor(case.block_table[b, : -(-(L + n) // P)].astype(np.int64), device=case.k_cache.device)
    both = []
    for pool, new in ((case.k_cache, case.k_new), (case.v_cache, case.v_new)):
        x = pool[pages]
        x = x if case.layout == wl.NHD else x.transpose(1, 2)
        x = x.reshape(-1, case.num_kv_heads, case.head_dim)[: L + n].double()
        if with_new:
            x[L:] = new[lo:lo + n].to(x.device).double()
        both.append(x)
    return both


def attention(case, seen_rows, with_new=True, rows=None):
    """out, lse in 64 bits, and the bound of a correct kernel's error in out.

    The bound: out is rounded to bf16 once (half a step, 2^-8 |out|).  Before
    that a key's weight is off by a relative delta: the score's products are
    exact in fp32 and summed over head_dim in fp32 (at most head_dim * 2^-24 of
    scale * sum |q k|, at most twice that through the base-2 scaling and the
    running maximum), exp2 is off by 2^-22 and the weight is kept in 16 bits or
    more (2^-17); with the sums over the keys in fp32 in any order another
    2^-17 covers 2^7 roundings in a row.  Weights off by delta, divided by their
    sum, move a weighted mean by at most 2 delta max |v| over the node's keys."""
    T, H, D = case.q.shape
    K = case.num_kv_heads
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -math.inf)
    tol = np.zeros((T, H, D))
    for b in rows if rows is not None else range(case.batch):
        lo, hi = int(case.qo_indptr[b]), int(case.qo_indptr[b + 1])
        n, L = hi - lo, int(case.cache_seqlens[b])
        if n == 0 or L < 0:
            continue
        k, v = row_kv(case, b, n, with_new)
        seen = torch.ones(n, L + n, dtype=torch.bool, device=k.device)
        seen[:, L:] = torch.as_tensor(seen_rows[b], device=k.device)
        q = case.q[lo:hi].to(k.device).double()
        for h in range(H):
            kg, vg = k[:, h // (H // K)], v[:, h // (H // K)]
            kg = torch.where(seen.any(0)[:, None], kg, 0.0)  # a key that no node sees may hold anything
            s = (q[:, h] @ kg.T) * case.softmax_scale
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(1, keepdim=True).nan_to_num(neginf=0.0)
            p = torch.exp(s - top)
            total = p.sum(1, keepdim=True)
            vv = torch.where(seen.any(0)[:, None], vg, 0.0)
            # a masked key's value never reaches the node, not even an infinite one
            finite = torch.isfinite(vv).all(1)
            o = p[:, finite] @ vv[finite]
            for j in torch.nonzero(~finite).flatten().tolist():
                o = torch.where(seen[:, j, None], o + p[:, j, None] * vv[j], o)
            o = o / torch.where(total == 0, 1.0, total)
            big = (q[:, h].abs() @ torch.where(torch.isfinite(kg), kg, 0.0).abs().T).amax(1, keepdim=True)
            delta = 2 * D * 2.0 ** -24 * abs(case.softmax_scale) * big + 2.0 ** -22 + 2.0 ** -17 + 2.0 ** -17
            out[lo:hi, h] = o.cpu().numpy()
            reach = torch.where(seen[:, finite], vv[finite].abs().amax(1), 0.0).amax(1, keepdim=True)
            tol[lo:hi, h] = (2.0 ** -8 * o.abs() + 2 * delta * reach).cpu().numpy()
            lse[lo:hi, h] = (top + total.log())[:, 0].cpu().numpy()
    return out, lse, tol


def accept(parents, draft, target, root, max_path):
    """Accepted path of one row, and the token after it (root None: the first
    node without a parent is taken unseen)."""
    path, cur = [], -1
    while len(path) < max_path:
        want = target[cur] if cur >= 0 else root
        kids = [i for i, p in enumerate(parents) if p == cur and (want is None or draft[i] == want)]
        if not kids:
            break
        cur = kids[0]
        path.append(cur)
    return path, (target[cur] if cur >= 0 else (-1 if root is None else root))


class TablePool:
    """The device pool and table update, a row and a block at a time."""

    def __init__(self, num_pages, batch, max_blocks, page_size, ring=None):
        self.free = list(ring if ring is not None else range(1, num_pages))  # head first
        self.page = page_size
        self.table = np.zeros((batch, max_blocks), np.int64)
        self.held = np.zeros(batch, np.int64)

    def update(self, lens, new, max_tokens=None):
        """indptr, slots, positions, failed rows ({row: why})."""
        P, (B, width) = self.page, self.table.shape
        failed, n, want, tokens = {}, [0] * B, list(self.held), 0
        for b in range(B):
            m = int(new[b]) if lens[b] >= 0 else 0
            need = -(-(int(lens[b]) + m) // P) if lens[b] >= 0 else 0
            if m < 0:
                failed[b] = "qlen"
            elif need > width:
                failed[b] = "overflow"
            else:
                tokens += m
                if max_tokens is not None and m > 0 and tokens > max_tokens:
                    failed[b] = "qlen"
                else:
                    n[b], want[b] = m, need
        asked = 0
        for b in range(B):
            if b not in failed and want[b] > self.held[b]:
                asked += want[b] - self.held[b]
                if asked > len(self.free):
                    failed[b], n[b], want[b] = "pool", 0, self.held[b]
        back = []
        for b in range(B):
            for k in range(int(self.held[b]), int(want[b])):
                self.table[b, k] = self.free.pop(0)
            for k in range(int(want[b]), int(self.held[b])):
                back.append(int(self.table[b, k]))
                self.table[b, k] = 0
            self.held[b] = want[b]
        self.free += back
        indptr = np.concatenate([[0], np.cumsum(n)])
        total = int(indptr[-1]) if max_tokens is None else max_tokens
        slots, pos = np.full(total, -1, np.int64), np.full(total, -1, np.int64)
        for b in range(B):
            for i in range(n[b]):
                at = int(lens[b]) + i
                slots[indptr[b] + i] = self.table[b, at // P] * P + at % P
                pos[indptr[b] + i] = at
        return indptr, slots, pos, failed
