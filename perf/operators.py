"""Speculative decoding with trees of drafted tokens over the paged cache, and
the block tables behind it: the cases that are measured, the operators' plain
forms in elementary torch operations, and the calls a user makes of the
library's kernels.

One step of such a decoder is, in this order:

* ``tables`` -- the block tables follow the rows' lengths (pages taken from
  and returned to a pool on the device), with the slot of every new token;
* ``build``  -- ancestor masks and positions from the drafted trees' parents;
* ``attn``   -- append of the drafted tokens, attention of every node over its
  row's cache and its ancestors;
* ``accept`` -- the longest path whose tokens the target model chose itself;
* ``commit`` -- the accepted tokens' K/V move to the front, in every layer.
"""
import math
import random

import numpy as np
import torch

own = False

# The device pool of pages, as an int32 tensor: word 0 the ring index of the
# next page handed out, word 1 the number of free pages, the ring from here.
POOL_HEAD = 16


def _lib():
    import paged_kv_decode_append_gb300 as pkv

    return pkv


# ------------------------------------------------------------------- cases


def listed():
    return [
        # one drafted token on a short cache of a tiny layer: latency alone
        dict(name="attn_one_token", op="attn", batch=4, heads=4, kv_heads=2, dim=64, page=16, layout="nhd", len_lo=1,
             len_hi=64, long=0, nodes_lo=1, nodes_hi=1, append=True, len_seed=1),
        # the ordinary step: the 32-row layer of the decode benchmark, 16-node trees
        dict(name="attn_trees_16", op="attn", batch=32, heads=32, kv_heads=8, dim=128, page=16, layout="nhd",
             len_lo=512, len_hi=1024, long=0, nodes_lo=16, nodes_hi=16, append=True, len_seed=2),
        # skewed lengths with one 32K-token row, trees of up to 64 nodes
        dict(name="attn_trees_64_skewed", op="attn", batch=64, heads=32, kv_heads=8, dim=128, page=16, layout="nhd",
             len_lo=128, len_hi=4096, long=32768, nodes_lo=40, nodes_hi=64, append=True, len_seed=4),
        # wide heads over HND pages, ragged trees, K/V cached by the caller
        dict(name="attn_d256_ragged", op="attn", batch=8, heads=48, kv_heads=6, dim=256, page=16, layout="hnd",
             len_lo=65, len_hi=2047, long=0, nodes_lo=1, nodes_hi=33, append=False, len_seed=5),
        # a decode step's tables: every row grows or shrinks by a few blocks
        dict(name="tables_step", op="tables", batch=64, page=16, len_lo=128, len_hi=4096, new_lo=1, new_hi=64,
             admit=False, len_seed=6),
        # admission: half of the rows bring whole prompts, the other half is released
        dict(name="tables_admit", op="tables", batch=1024, page=16, len_lo=0, len_hi=0, new_lo=64, new_hi=1023,
             admit=True, len_seed=7),
        # masks of small trees, and of the largest trees at the largest batch
        dict(name="build_small", op="build", batch=4, nodes_lo=5, nodes_hi=8, len_seed=8),
        dict(name="build_large", op="build", batch=1024, nodes_lo=129, nodes_hi=256, len_seed=9),
        # acceptance over a few small trees, and over many of odd sizes
        dict(name="accept_small", op="accept", batch=4, nodes_lo=5, nodes_hi=8, len_seed=10),
        dict(name="accept_large", op="accept", batch=1024, nodes_lo=33, nodes_hi=129, len_seed=11),
        # accepted tokens of one small layer, and of the 36 layers of the batch sweep's model
        dict(name="commit_small", op="commit", layers=1, batch=4, kv_heads=2, dim=64, page=16, layout="nhd", len_lo=1,
             len_hi=64, nodes_lo=4, nodes_hi=8, len_seed=12),
        dict(name="commit_36_layers", op="commit", layers=36, batch=64, kv_heads=8, dim=128, page=128, layout="nhd",
             len_lo=64, len_hi=200, nodes_lo=16, nodes_hi=64, len_seed=13),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _span(rng, lo, hi):
    a, b = _log_int(rng, lo, hi), _log_int(rng, lo, hi)
    return min(a, b), max(a, b)


def draw(rng):
    op = rng.choice(["attn", "attn", "tables", "build", "accept", "commit"])
    c = dict(op=op, len_seed=rng.randrange(1 << 20))
    if op == "attn":
        c["batch"] = _log_int(rng, 1, 64)
        c["heads"], c["kv_heads"] = rng.choice([(4, 2), (32, 8), (48, 6), (8, 8), (16, 1), (24, 8)])
        c["dim"] = rng.choice([64, 128, 256])
        c["page"] = rng.choice([8, 16, 32, 64, 128, 256])
        c["layout"] = rng.choice(["nhd", "hnd"])
        c["len_lo"], c["len_hi"] = _span(rng, 1, 4096)
        c["long"] = rng.choice([0, 0, _log_int(rng, 4096, 32768)])
        c["nodes_lo"], c["nodes_hi"] = _span(rng, 1, 128)
        c["append"] = rng.random() < 0.7
        top = listed()[2]
        most = work(top)
        pad = max(top["long"], top["len_hi"]) * top["batch"]
        while True:  # no dearer than the largest listed case, in its work and in the plain form's padding
            w, keys = work(c), (max(c["long"], c["len_hi"]) + c["nodes_hi"]) * c["batch"]
            if (w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"]
                    and keys * c["heads"] * c["nodes_hi"] <= pad * top["heads"] * 64
                    and keys * c["kv_heads"] * c["dim"] <= pad * top["kv_heads"] * top["dim"]):
                return c
            c["batch"], c["len_hi"] = max(1, c["batch"] * 3 // 4), max(c["len_lo"], c["len_hi"] * 3 // 4)
            c["long"] = c["long"] * 3 // 4
            c["nodes_hi"] = max(c["nodes_lo"], c["nodes_hi"] * 7 // 8)
    if op == "tables":
        c["batch"] = _log_int(rng, 1, 1024)
        c["page"] = rng.choice([1, 8, 16, 64, 256])
        c["admit"] = rng.random() < 0.5
        c["len_lo"], c["len_hi"] = (0, 0) if c["admit"] else _span(rng, 1, 4096)
        c["new_lo"], c["new_hi"] = _span(rng, 1, 1023) if c["admit"] else _span(rng, 1, 256)
        while c["page"] < 16 and c["batch"] * (c["len_hi"] + c["new_hi"]) > 300000:
            c["batch"] = max(1, c["batch"] // 2)
        return c
    if op in ("build", "accept"):
        c["batch"] = _log_int(rng, 1, 1024)
        c["nodes_lo"], c["nodes_hi"] = _span(rng, 1, 256 if op == "build" else 129)
        return c
    c["layers"] = _log_int(rng, 1, 36)
    c["batch"] = _log_int(rng, 1, 64)
    c["kv_heads"] = rng.choice([1, 2, 6, 8])
    c["dim"] = rng.choice([64, 128])
    c["page"] = rng.choice([1, 8, 16, 64, 128])
    c["layout"] = rng.choice(["nhd", "hnd"])
    c["len_lo"], c["len_hi"] = _span(rng, 1, 128)
    c["nodes_lo"], c["nodes_hi"] = _span(rng, 1, 64)
    return c


def _lens(case):
    """Cached tokens of every row: uniform, or lognormal with one long row."""
    r = random.Random(case["len_seed"])
    lo, hi = case["len_lo"], case["len_hi"]
    if case.get("long"):
        lens = [min(hi, max(lo, int(r.lognormvariate(6.5, 0.8)))) for _ in range(case["batch"])]
        lens[0] = case["long"]
        return lens
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _counts(case, lo="nodes_lo", hi="nodes_hi"):
    """Drafted (or new) tokens of every row."""
    r = random.Random(case["len_seed"] + 77)
    return [r.randint(case[lo], case[hi]) for _ in range(case["batch"])]


def _table_turns(case):
    """The two lists of (cached, new) tokens that a tables case turns between:
    admission lets one half of the rows in and the other out; a decode step's
    rows move by up to four blocks."""
    lens, new = _lens(case), _counts(case, "new_lo", "new_hi")
    if case["admit"]:
        return [[(0, n) if (b + t) % 2 == 0 else (-1, 0) for b, n in enumerate(new)] for t in (0, 1)]
    r = random.Random(case["len_seed"] + 5)
    shift = [r.randint(-4 * case["page"], 4 * case["page"]) for _ in lens]
    return [[(max(0, L + (s if t else 0)), n) for L, n, s in zip(lens, new, shift)] for t in (0, 1)]


def work(case):
    op, B = case["op"], case["batch"]
    if op == "tables":
        total = {"bytes": 0.0, "flops": 0.0}
        turns, P = _table_turns(case), case["page"]
        blocks = [[0 if L < 0 else -(-(L + n) // P) for L, n in t] for t in turns]
        for t, have, want in ((0, blocks[1], blocks[0]), (1, blocks[0], blocks[1])):
            moved = sum(abs(a - b) for a, b in zip(have, want))
            gone = sum(max(0, a - b) for a, b in zip(have, want))
            tokens = sum(n for _, n in turns[t])
            # lengths, counts, prefix; page ids read and written (and zeroed); a slot and a position for each token
            total["bytes"] += (4 * (3 * B + 2 * B + 1) + 8 * moved + 4 * gone + 12 * tokens) / 2
        return total
    n = _counts(case)
    T = sum(n)
    words = -(-case["nodes_hi"] // 32)
    if op == "build":
        return {"bytes": 4.0 * (2 * B + 1) + T * (4.0 + 4 * words + 4), "flops": 0.0}
    if op == "accept":
        return {"bytes": 4.0 * (3 * B + 1) + 12.0 * T + 4.0 * B * (case["nodes_hi"] + 3), "flops": 0.0}
    if op == "commit":
        # half of a tree's depth or so is accepted: see _tokens(); K and V of each, read and written
        kept = sum(_kept(case))
        return {"bytes": 4.0 * (2 * B + kept * 3) + case["layers"] * kept * 8.0 * case["kv_heads"] * case["dim"],
                "flops": 0.0}
    lens = _lens(case)
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    keys = sum(lens) + (0 if case["append"] else T)
    b = 4.0 * keys * K * D + (8.0 * T * K * D if case["append"] else 0.0)      # K and V cached; new ones read and written
    b += 4.0 * T * H * D + 4.0 * T * H + 4.0 * T * words                       # q, out, lse, masks
    b += 4.0 * sum(-(-(L + m) // case["page"]) for L, m in zip(lens, n)) + 4.0 * (2 * B + 1)
    seen = sum(m * L + m * math.log2(m + 1) for L, m in zip(lens, n))          # a random tree's depth is about its logarithm
    return {"bytes": b, "flops": 4.0 * D * H * seen}


# ------------------------------------------------------------------- inputs


def _tree_parents(counts, seed):
    """Random recursive trees: a node's parent is any earlier node, or the cache (-1)."""
    r = np.random.RandomState(seed % (1 << 31))
    return [np.floor(r.rand(n) * (np.arange(n) + 1)).astype(np.int64) - 1 for n in counts]


def _masks(parents, words):
    """Ancestor bits of every node, as int32 words."""
    rows = []
    for p in parents:
        seen = np.eye(len(p), words * 32, dtype=bool)
        for i, up in enumerate(p):
            if up >= 0:
                seen[i] |= seen[up]
        rows.append(np.packbits(seen, axis=1, bitorder="little").view(np.int32))
    return np.concatenate(rows)


def _tokens(parents, seed):
    """Drafted tokens, the target model's choice after every node, and after
    the cached tokens: about three in four of the inner nodes have a child
    that the target chose."""
    r = np.random.RandomState((seed + 1) % (1 << 31))
    drafts, targets, roots = [], [], []
    for p in parents:
        n = len(p)
        d = r.randint(0, 150000, n)
        t = np.concatenate([[r.randint(0, 150000)], r.randint(0, 150000, n)])
        take = r.rand(n) < 0.75
        t[p[take] + 1] = d[take]
        drafts.append(d)
        targets.append(t[1:])
        roots.append(t[0])
    return np.concatenate(drafts), np.concatenate(targets), np.array(roots)


def _indptr(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device="cuda")


def _pages(case, tokens, g):
    """A block table whose rows hold `tokens` tokens each, on shuffled pages."""
    need = [-(-t // case["page"]) for t in tokens]
    num_pages = sum(need) * 5 // 4 + 8
    ids = torch.randperm(num_pages - 1, generator=g, device="cuda").to(torch.int32) + 1
    width = max(max(need), 1)
    k = torch.arange(width, device="cuda")
    n, first = torch.as_tensor(need, device="cuda")[:, None], torch.as_tensor(_indptr(need)[:-1], device="cuda")[:, None]
    table = torch.where(k < n, ids[(first + k).clamp_(max=num_pages - 2)], 0)
    return num_pages, table.to(torch.int32).contiguous()


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _kept(case):
    """Accepted tokens of every row of a commit case."""
    r = random.Random(case["len_seed"] + 3)
    return [r.randint(0, min(m, 8)) for m in _counts(case)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, B = case["op"], case["batch"]
    s = {"case": case, "op": op}
    if op == "tables":
        P, turns = case["page"], _table_turns(case)
        most = [max(t[b][0] + t[b][1] for t in turns) for b in range(B)]
        width = max(1, max(-(-max(0, m) // P) for m in most))
        pages = 2 * sum(-(-max(0, m) // P) for m in most) + 8
        ring = torch.randperm(pages, generator=g, device="cuda").to(torch.int32) + 1
        head = torch.zeros(POOL_HEAD, dtype=torch.int32, device="cuda")
        head[1] = pages
        s["pool"] = torch.cat([head, ring])
        s["table"] = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        s["held"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["turns"] = [(_i32([L for L, _ in t]), _i32([n for _, n in t])) for t in turns]
        s["max_tokens"] = max(sum(n for _, n in t) for t in turns)
        s["turn"] = 0
        s["indptr"] = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(s["max_tokens"], dtype=torch.int64, device="cuda")
        s["positions"] = torch.empty(s["max_tokens"], dtype=torch.int32, device="cuda")
        return s
    counts = _counts(case)
    parents = _tree_parents(counts, seed)
    s["counts_max"] = case["nodes_hi"]
    s["words"] = -(-case["nodes_hi"] // 32)
    s["indptr"] = _i32(_indptr(counts))
    T = sum(counts)
    if op in ("build", "accept"):
        s["parents"] = _i32(np.concatenate(parents))
        s["seqlens"] = torch.randint(0, 4096, (B,), generator=g, device="cuda").to(torch.int32)
        if op == "build":
            s["mask"] = torch.empty(T, s["words"], dtype=torch.int32, device="cuda")
            s["positions"] = torch.empty(T, dtype=torch.int32, device="cuda")
        else:
            s["draft"], s["target"], s["root"] = (_i32(x) for x in _tokens(parents, seed))
            s["path"] = torch.empty(B, case["nodes_hi"], dtype=torch.int32, device="cuda")
            s["length"], s["next"], s["after"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
        return s
    lens = _lens(case)
    s["seqlens"] = _i32(lens)
    pages, s["table"] = _pages(case, [L + n for L, n in zip(lens, counts)], g)
    K, D, P = case["kv_heads"], case["dim"], case["page"]
    shape = (pages, P, K, D) if case["layout"] == "nhd" else (pages, K, P, D)
    if op == "commit":
        kept = _kept(case)
        r = np.random.RandomState(seed % (1 << 31))
        path = np.full((B, max(1, max(kept))), -1)
        for b, (n, k) in enumerate(zip(counts, kept)):
            path[b, :k] = np.sort(r.permutation(n)[:k])
        s["path"], s["length"] = _i32(path), _i32(kept)
        s["k"] = _normal((case["layers"],) + shape, g)
        s["v"] = _normal((case["layers"],) + shape, g)
        return s
    H = case["heads"]
    s["k"], s["v"], s["q"] = _normal(shape, g), _normal(shape, g), _normal((T, H, D), g)
    s["k_new"], s["v_new"] = (_normal((T, K, D), g), _normal((T, K, D), g)) if case["append"] else (None, None)
    s["mask"] = torch.as_tensor(_masks(parents, s["words"]), device="cuda")
    s["scale"] = 1.0 / math.sqrt(D)
    s["keys_max"] = max(L + n for L, n in zip(lens, counts))
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------- one pass


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _rows_of(indptr, T):
    """Row and index within the row of every token."""
    t = torch.arange(T, device="cuda")
    row = torch.searchsorted(indptr[1:].long(), t, right=True).clamp_(max=indptr.numel() - 2)
    return row, t - indptr.long()[row]


def _padded_rows(indptr, n):
    """For [row, node] of a padded batch: the token, and whether there is one."""
    i = torch.arange(n, device="cuda")
    first, count = indptr[:-1].long()[:, None], (indptr[1:] - indptr[:-1]).long()[:, None]
    live = i < count
    return torch.where(live, first + i, 0), live


def _plain_tables(s):
    lens, new = s["turns"][s["turn"]]
    s["turn"] ^= 1
    pool, table, held, P = s["pool"], s["table"], s["held"].long(), s["case"]["page"]
    ring, room = pool[POOL_HEAD:], pool.numel() - POOL_HEAD
    lens, new = lens.long(), torch.where(lens < 0, 0, new).long()
    want = torch.where(lens < 0, 0, (lens + new + P - 1) // P)
    take, give = (want - held).clamp(min=0), (held - want).clamp(min=0)
    took, gave = take.cumsum(0), give.cumsum(0)
    head, count = pool[0].long(), pool[1].long()
    k = torch.arange(table.shape[1], device="cuda")
    at = (head + (took - take)[:, None] + k - held[:, None]) % room
    fresh = (k >= held[:, None]) & (k < want[:, None])
    gone = (k >= want[:, None]) & (k < held[:, None])
    # a returned page's place in the ring; entries that stay go to a place behind it
    to = torch.where(gone, (head + count + (gave - give)[:, None] + k - want[:, None]) % room, room)
    longer = torch.cat([ring, ring[:1]])
    found = torch.where(fresh, ring[at], table)
    longer[to.view(-1)] = torch.where(gone, table, 0).view(-1)
    ring.copy_(longer[:room])
    table.copy_(torch.where(gone, 0, found))
    pool[0] = ((head + took[-1]) % room).int()
    pool[1] = (count - took[-1] + gave[-1]).int()
    s["held"].copy_(want)
    indptr = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)]).int()
    T = s["max_tokens"]
    row, i = _rows_of(indptr, T)
    live = torch.arange(T, device="cuda") < indptr[-1]
    at = torch.where(live, lens[row] + i, 0)
    slots = table[row, at // P].long() * P + at % P
    return {"pool": pool, "table": table, "held": s["held"], "indptr": indptr, "slots": torch.where(live, slots, -1),
            "positions": torch.where(live, at, -1).int()}


def _own_tables(s):
    lens, new = s["turns"][s["turn"]]
    s["turn"] ^= 1
    _lib().pkv_table_update(s["pool"], s["table"], s["held"], lens, new, s["case"]["page"], indptr=s["indptr"],
                            slot_map=s["slots"], positions=s["positions"])
    return {"pool": s["pool"], "table": s["table"], "held": s["held"], "indptr": s["indptr"], "slots": s["slots"],
            "positions": s["positions"]}


def _padded_parents(s):
    n = s["counts_max"]
    tok, live = _padded_rows(s["indptr"], n)
    return tok, live, torch.where(live, s["parents"].long()[tok], -1)


def _plain_build(s):
    n, words = s["counts_max"], s["words"]
    tok, live, up = _padded_parents(s)
    B = up.shape[0]
    # bits of ancestors by pointer doubling; a last, empty node stands for the cache
    seen = torch.zeros(B, n + 1, words * 32, dtype=torch.bool, device="cuda")
    seen[:, :n, :n] = torch.eye(n, dtype=torch.bool, device="cuda")
    up = torch.cat([torch.where(up < 0, n, up), torch.full_like(up[:, :1], n)], 1)
    for _ in range(max(1, (n - 1).bit_length())):
        seen = seen | torch.gather(seen, 1, up[:, :, None].expand(-1, -1, words * 32))
        up = torch.gather(up, 1, up)
    depth = seen.sum(2) - 1
    bits = 2 ** torch.arange(32, device="cuda")
    packed = (seen.view(B, n + 1, words, 32) * bits).sum(3)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
    row, i = _rows_of(s["indptr"], s["parents"].numel())
    return {"mask": packed[row, i], "positions": (s["seqlens"].long()[row] + depth[row, i]).int()}


def _own_build(s):
    _lib().pkv_tree_build(s["parents"], s["indptr"], s["seqlens"], s["counts_max"], mask=s["mask"],
                          positions=s["positions"])
    return {"mask": s["mask"], "positions": s["positions"]}


def _plain_attn(s):
    c = s["case"]
    H, K, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    G, B, n, L = H // K, c["batch"], s["counts_max"], s["seqlens"].long()
    k, v = (x if c["layout"] == "nhd" else x.transpose(1, 2) for x in (s["k"], s["v"]))
    table = s["table"].long()
    row, i = _rows_of(s["indptr"], s["q"].shape[0])
    if s["k_new"] is not None:
        at = L[row] + i
        page = table[row, at // P]
        k[page, at % P] = s["k_new"]
        v[page, at % P] = s["v_new"]
    at = torch.arange(s["keys_max"], device="cuda")
    page = table[:, (at // P).clamp(max=table.shape[1] - 1)]
    keys = k[page, at % P].permute(0, 2, 3, 1).float()                                        # [B, K, D, keys]
    values = v[page, at % P].permute(0, 2, 1, 3).float()                                      # [B, K, keys, D]
    tok, live = _padded_rows(s["indptr"], n)
    q = s["q"][tok].float().view(B, n, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, n * G, D)
    scores = (q @ keys).mul_(s["scale"]).view(B, K, n, G, -1)
    j = at - L[:, None]                                                                       # drafted key, or below 0
    bit = s["mask"][tok].gather(2, (j.clamp(0, n - 1) // 32)[:, None].expand(B, n, -1)) >> (j.clamp(min=0) % 32)[:, None]
    count = live.sum(1)[:, None, None]
    seen = (j[:, None] < 0) | ((j[:, None] < count) & ((bit & 1) == 1))
    scores = scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, K, n * G, -1) @ values).view(B, K, n, G, D) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0]
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, n, H, D)[row, i].to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, n, H)[row, i], "k": s["k"], "v": s["v"]}


def _own_attn(s):
    pkv = _lib()
    c = s["case"]
    layout = pkv.NHD if c["layout"] == "nhd" else pkv.HND
    if "workspace" not in s:
        s["workspace"] = pkv.tree_workspace(c["batch"], s["q"].shape[0], s["table"].shape[1], c["heads"],
                                            s["counts_max"], pkv.cache_desc(s["k"], layout), s["q"].device)
    pkv.pkv_tree_attn(s["k"], s["v"], s["q"], s["k_new"], s["v_new"], s["indptr"], s["mask"], s["table"], s["seqlens"],
                      s["scale"], s["counts_max"], out=s["out"], lse=s["lse"], workspace=s["workspace"], layout=layout)
    return {"out": s["out"], "lse": s["lse"], "k": s["k"], "v": s["v"]}


def _plain_accept(s):
    n = s["counts_max"]
    tok, live, up = _padded_parents(s)
    draft, target = s["draft"].long()[tok], s["target"].long()[tok]
    want = torch.cat([s["root"].long()[:, None], target], 1).gather(1, up + 1)
    good = live & (draft == want)
    i = torch.arange(n, device="cuda").expand_as(up)
    # of a node's children that fit, the first
    first = torch.full((up.shape[0], n + 1), n, dtype=torch.int64, device="cuda")
    first.scatter_reduce_(1, up + 1, torch.where(good, i, n), "amin")
    good = good & (first.gather(1, up + 1) == i)
    # a node counts when its ancestors do: pointer doubling, the last place stands for the cache
    good = torch.cat([good, torch.ones_like(good[:, :1])], 1)
    hop = torch.cat([torch.where(up < 0, n, up), torch.full_like(up[:, :1], n)], 1)
    for _ in range(max(1, (n - 1).bit_length())):
        good = good & torch.gather(good, 1, hop)
        hop = torch.gather(hop, 1, hop)
    good = good[:, :n]
    length = good.sum(1)
    at = torch.where(good, good.long().cumsum(1) - 1, n)
    path = torch.full((up.shape[0], n + 1), -1, dtype=torch.int64, device="cuda").scatter_(1, at, i)[:, :n]
    path = torch.where(i < length[:, None], path, -1)
    last = path.gather(1, (length - 1).clamp(min=0)[:, None])
    after = torch.cat([s["root"].long()[:, None], target], 1).gather(1, last + 1)[:, 0]
    return {"path": path.int(), "length": length.int(), "next": after.int(),
            "after": (s["seqlens"].long() + length).int()}


def _own_accept(s):
    _lib().pkv_tree_accept(s["parents"], s["draft"], s["target"], s["root"], s["indptr"], s["seqlens"], s["counts_max"],
                           path=s["path"], path_len=s["length"], next_token=s["next"], seqlens_out=s["after"])
    return {"path": s["path"], "length": s["length"], "next": s["next"], "after": s["after"]}


def _plain_commit(s):
    P, nhd = s["case"]["page"], s["case"]["layout"] == "nhd"
    k, v = (x if nhd else x.transpose(2, 3) for x in (s["k"], s["v"]))
    table, path, L = s["table"].long(), s["path"].long(), s["seqlens"].long()[:, None]
    i = torch.arange(path.shape[1], device="cuda").expand_as(path)
    # a row's unused places copy its slots onto themselves: of the last accepted token, or of position 0
    length = s["length"].long()[:, None]
    spare = torch.where(length > 0, L + length - 1, 0)
    tail = path.gather(1, (length - 1).clamp(min=0))
    src = torch.where(i < length, L + path, torch.where(length > 0, L + tail, 0))
    dst = torch.where(i < length, L + i, spare)
    row = torch.arange(path.shape[0], device="cuda")[:, None]
    for x in (k, v):
        x[:, table[row, dst // P], dst % P] = x[:, table[row, src // P], src % P]
    return {"k": s["k"], "v": s["v"]}


def _own_commit(s):
    pkv = _lib()
    if "layers" not in s:
        s["layers"] = pkv.LayerCaches(list(s["k"]), list(s["v"]), pkv.NHD if s["case"]["layout"] == "nhd" else pkv.HND)
    pkv.pkv_tree_commit(s["layers"], s["path"], s["length"], s["table"], s["seqlens"])
    return {"k": s["k"], "v": s["v"]}


_plain = {"tables": _plain_tables, "build": _plain_build, "attn": _plain_attn, "accept": _plain_accept,
          "commit": _plain_commit}
_own = {"tables": _own_tables, "build": _own_build, "attn": _own_attn, "accept": _own_accept, "commit": _own_commit}


# ------------------------------------------------------------------- 64 bits


def exact(case, seed):
    """Row by row and head by head in 64 bits; the other operators move or
    count whole values only."""
    if case["op"] == "commit":
        return _exact_commit(case, seed)
    if case["op"] != "attn":
        return None
    s = prepare(case, seed)
    lens, first = _lens(case), _indptr(_counts(case))
    H, K, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    bits = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    bits = bits.flatten(1).bool()
    for b, L in enumerate(lens):
        lo, hi = int(first[b]), int(first[b + 1])
        n = hi - lo
        pages = s["table"][b, : -(-(L + n) // P)].long()
        both = []
        for pool, fresh in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
            x = pool[pages]
            x = (x if case["layout"] == "nhd" else x.transpose(1, 2)).reshape(-1, K, D)[: L + n].double()
            if fresh is not None:
                x[L:] = fresh[lo:hi].double()
            both.append(x)
        seen = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
        seen[:, L:] = bits[lo:hi, :n]
        for h in range(H):
            g = h // (H // K)
            a = s["q"][lo:hi, h].double() @ both[0][:, g].T * s["scale"]
            a = a.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(a, 1)
            lse[lo:hi, h] = z
            out[lo:hi, h] = torch.exp(a - z[:, None]) @ both[1][:, g]
    return {"out": out, "lse": lse, "k": None, "v": None}


def _exact_commit(case, seed):
    s = prepare(case, seed)
    P, lens = case["page"], _lens(case)
    table, path = s["table"].tolist(), s["path"].tolist()
    src, dst = [], []
    for b, kept in enumerate(_kept(case)):
        for i in range(kept):
            for where, at in ((src, lens[b] + path[b][i]), (dst, lens[b] + i)):
                where.append((table[b][at // P], at % P))
    got = {}
    for name in ("k", "v"):
        x = s[name].double()
        y = x if case["layout"] == "nhd" else x.transpose(2, 3)
        if src:
            a, b = (torch.tensor(w, device="cuda").T for w in (src, dst))
            y[:, b[0], b[1]] = y[:, a[0], a[1]]
        got[name] = x
    return got
