"""A paged cache kept inside a budget by accumulated attention weight, and the
rotary positions that this asks for: the cases that are measured, the
operators' plain forms in elementary torch operations, and the calls a user
makes of the library's kernels.

One step of such a decoder is, in this order:

* ``rope``  -- queries and new keys rotated by their tokens' positions (after an
  eviction no longer their slots), new K/V appended to the cache;
* ``mass``  -- after the attention, whose log-sum-exps it takes: what the
  step's queries give to every cached token, added up per kv head;
* ``plan``  -- the slots that a row keeps, for every layer and kv head on their
  own, and the moves that fill the holes in front;
* ``apply`` -- the moves: K, V, scores and positions, and the rows' lengths.
"""
import math
import random

import numpy as np
import torch

own = False


def _lib():
    import paged_kv_decode_append_gb300 as pkv

    return pkv


# ------------------------------------------------------------------- cases


def listed():
    return [
        # one new token for each row of a tiny layer: latency alone
        dict(name="rope_one_token", op="rope", batch=4, heads=4, kv_heads=2, dim=64, rot=64, pairing="half", page=16,
             layout="nhd", len_lo=1, len_hi=64, new_lo=1, new_hi=1, chunks=0, gone=0, scaling="none", append=True, len_seed=1),
        # the chunked-prefill step of the decode benchmark's layer, context stretched by parts
        dict(name="rope_chunked_step", op="rope", batch=64, heads=32, kv_heads=8, dim=128, rot=128, pairing="half", page=16,
             layout="nhd", len_lo=512, len_hi=2048, new_lo=1, new_hi=1, chunks=496, gone=30000, scaling="parts", append=True,
             len_seed=2),
        # whole prompts of the wide ragged-prefill heads, a quarter of each rotated, neighbours as pairs
        dict(name="rope_prompts_partial", op="rope", batch=16, heads=48, kv_heads=6, dim=256, rot=64, pairing="interleaved",
             page=16, layout="hnd", len_lo=0, len_hi=2047, new_lo=65, new_hi=1023, chunks=0, gone=0, scaling="linear",
             append=True, len_seed=3),
        # a decode step of a tiny layer: latency alone
        dict(name="mass_one_token", op="mass", batch=4, heads=4, kv_heads=2, dim=64, page=16, layout="nhd", len_lo=1,
             len_hi=64, long=0, new_lo=1, new_hi=1, fresh="new", len_seed=4),
        # a decode step over skewed lengths, one row of 32K tokens
        dict(name="mass_decode_skewed", op="mass", batch=64, heads=32, kv_heads=8, dim=128, page=16, layout="nhd",
             len_lo=128, len_hi=4096, long=32768, new_lo=1, new_hi=1, fresh="new", len_seed=5),
        # scores of prompts from their last queries alone
        dict(name="mass_window", op="mass", batch=8, heads=32, kv_heads=8, dim=128, page=128, layout="nhd", len_lo=2000,
             len_hi=8100, long=0, new_lo=16, new_hi=33, fresh="all", len_seed=6),
        # every query of two long prompt chunks
        dict(name="mass_prompts", op="mass", batch=2, heads=32, kv_heads=8, dim=128, page=16, layout="nhd", len_lo=500,
             len_hi=2047, long=0, new_lo=3500, new_hi=4095, fresh="new", len_seed=7),
        # ragged prompts of wide heads over HND pages
        dict(name="mass_prompts_d256", op="mass", batch=8, heads=48, kv_heads=6, dim=256, page=16, layout="hnd", len_lo=0,
             len_hi=2047, long=0, new_lo=65, new_hi=1023, fresh="new", len_seed=8),
        # one layer's rows over budget by a few tokens
        dict(name="plan_small", op="plan", layers=1, batch=4, kv_heads=2, len_lo=40, len_hi=64, budget=32, sink=4, recent=8,
             len_seed=9),
        # all 36 layers of a full batch, 64 tokens over a budget of 2048
        dict(name="plan_36_layers", op="plan", layers=36, batch=64, kv_heads=8, len_lo=2049, len_hi=2112, budget=2048,
             sink=4, recent=256, len_seed=10),
        # the moves of the tiny layer's rows
        dict(name="apply_small", op="apply", layers=1, batch=4, kv_heads=2, dim=64, page=16, layout="nhd", len_lo=40,
             len_hi=64, budget=32, sink=4, recent=8, len_seed=11),
        # prompts cut down to half their tokens, in all 36 layers
        dict(name="apply_36_layers", op="apply", layers=36, batch=8, kv_heads=8, dim=128, page=16, layout="nhd", len_lo=900,
             len_hi=1100, budget=500, sink=4, recent=64, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _span(rng, lo, hi):
    a, b = _log_int(rng, lo, hi), _log_int(rng, lo, hi)
    return min(a, b), max(a, b)


def draw(rng):
    op = rng.choice(["rope", "mass", "mass", "plan", "apply"])
    c = dict(op=op, len_seed=rng.randrange(1 << 20))
    most = max((work(x) for x in listed() if x["op"] == op), key=lambda w: w["bytes"])
    if op in ("rope", "mass"):
        c["heads"], c["kv_heads"] = rng.choice([(4, 2), (32, 8), (48, 6), (8, 8), (16, 1), (24, 8)])
        c["dim"] = rng.choice([64, 128, 256])
        c["page"] = rng.choice([8, 16, 32, 64, 128, 256])
        c["layout"] = rng.choice(["nhd", "hnd"])
        c["batch"] = _log_int(rng, 1, 64)
        c["len_lo"], c["len_hi"] = _span(rng, 1, 4096)
    if op == "rope":
        c["rot"] = rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= c["dim"]])
        c["pairing"] = rng.choice(["half", "interleaved"])
        c["new_lo"], c["new_hi"] = _span(rng, 1, 1023)
        c["chunks"] = rng.choice([0, 0, _log_int(rng, 16, 1023)])
        c["gone"] = rng.choice([0, _log_int(rng, 1, 1000000)])
        c["scaling"] = rng.choice(["none", "linear", "parts"])
        c["append"] = rng.random() < 0.7
        while work(c)["bytes"] > most["bytes"] or c["batch"] * (c["len_hi"] + c["new_hi"]) > 100000:
            c["batch"], c["new_hi"] = max(1, c["batch"] * 3 // 4), max(c["new_lo"], c["new_hi"] * 3 // 4)
            c["len_hi"] = max(c["len_lo"], c["len_hi"] * 3 // 4)
            if c["batch"] == 1:
                c["new_lo"] = max(1, c["new_lo"] * 3 // 4)
        return c
    if op == "mass":
        c["long"] = rng.choice([0, 0, _log_int(rng, 4096, 32768)])
        kind = rng.choice(["decode", "window", "prompt"])
        c["new_lo"], c["new_hi"] = (1, 1) if kind == "decode" else _span(rng, 1, 64) if kind == "window" else _span(rng, 64, 4095)
        c["fresh"] = rng.choice(["new", "all"])
        top = [x for x in listed() if x["name"] == "mass_prompts"][0]
        skew = [x for x in listed() if x["name"] == "mass_decode_skewed"][0]
        flops, bytes_ = work(top)["flops"], work(skew)["bytes"]
        while True:  # no dearer than the listed ones, in its work and in the plain form's padding
            w, keys = work(c), (max(c["long"], c["len_hi"]) + c["new_hi"]) * c["batch"]
            if (w["flops"] <= flops and w["bytes"] <= bytes_ and keys * c["heads"] * c["new_hi"] <= 2 * 6142 * 32 * 4095
                    and keys * c["kv_heads"] * c["dim"] <= 32768 * 64 * 8 * 128):
                return c
            c["batch"], c["len_hi"] = max(1, c["batch"] * 3 // 4), max(c["len_lo"], c["len_hi"] * 3 // 4)
            c["long"] = c["long"] * 3 // 4
            c["new_hi"] = max(c["new_lo"], c["new_hi"] * 7 // 8)
            if c["batch"] == 1 and c["new_hi"] == c["new_lo"]:
                c["new_lo"] = c["new_hi"] = max(1, c["new_lo"] * 7 // 8)
    c["kv_heads"] = rng.choice([1, 2, 6, 8])
    c["layers"] = _log_int(rng, 1, 36)
    c["sink"] = rng.choice([0, 1, 4, 16])
    c["batch"] = _log_int(rng, 1, 64)
    if op == "plan":
        c["len_lo"], c["len_hi"] = _span(rng, 1, 32768)
    else:
        c["dim"] = rng.choice([64, 128, 256])
        c["page"] = rng.choice([1, 8, 16, 64, 256])
        c["layout"] = rng.choice(["nhd", "hnd"])
        c["len_lo"], c["len_hi"] = _span(rng, 1, 2048)
    c["budget"] = _log_int(rng, 1, c["len_hi"])
    c["recent"] = rng.randint(0, max(0, c["budget"] - c["sink"]))
    while True:
        slots = c["layers"] * c["batch"] * c["kv_heads"] * c["len_hi"]
        if work(c)["bytes"] <= most["bytes"] and slots * (1 if op == "plan" else c["dim"]) <= (4e7 if op == "plan" else 3.2e8):
            return c
        c["batch"], c["layers"] = max(1, c["batch"] * 3 // 4), max(1, c["layers"] * 7 // 8)
        if c["batch"] * c["layers"] == 1:
            c["len_hi"] = max(1, c["len_hi"] * 3 // 4)
            c["len_lo"], c["budget"] = min(c["len_lo"], c["len_hi"]), min(c["budget"], c["len_hi"])
            c["recent"] = min(c["recent"], max(0, c["budget"] - c["sink"]))


def _lens(case):
    """Cached tokens of every row: uniform, or lognormal with one long row."""
    r = random.Random(case["len_seed"])
    lo, hi = case["len_lo"], case["len_hi"]
    if case.get("long"):
        lens = [min(hi, max(lo, int(r.lognormvariate(6.5, 0.8)))) for _ in range(case["batch"])]
        lens[0] = case["long"]
        return lens
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _counts(case):
    """New tokens of every row; with `chunks`, four rows bring a chunk of a prompt."""
    r = random.Random(case["len_seed"] + 77)
    n = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    if case.get("chunks"):
        n[:4] = [case["chunks"]] * min(4, case["batch"])
    return n


def _need(case):
    """For rows of a plan: (length, slots kept, moves at most)."""
    lens = _lens(case)
    kept = [min(L, case["budget"]) for L in lens]
    return lens, kept, [min(k, L - k) for L, k in zip(lens, kept)]


def work(case):
    op, B = case["op"], case["batch"]
    if op == "rope":
        T = sum(_counts(case))
        heads = case["heads"] + (2 if case["append"] else 1) * case["kv_heads"]
        angles = 4.0 * case["rot"]                                                # a table of frequencies
        rows = 4.0 * (3 * B + 1) + 4.0 * T // case["page"] if case["append"] else 4.0 * T
        return {"bytes": T * heads * case["dim"] * 4.0 + rows + angles,
                "flops": 3.0 * T * (case["heads"] + case["kv_heads"]) * case["rot"]}
    if op == "mass":
        lens, n, H, K, D = _lens(case), _counts(case), case["heads"], case["kv_heads"], case["dim"]
        T, keys = sum(n), sum(lens) + sum(n)
        old = sum(lens) if case["fresh"] == "new" else 0
        b = 2.0 * keys * K * D + 2.0 * T * H * D + 4.0 * T * H                     # K, q, lse
        b += 4.0 * K * (old + keys) + 4.0 * K * (keys - old)                       # scores read and written; new positions
        b += 4.0 * sum(-(-(L + m) // case["page"]) for L, m in zip(lens, n)) + 4.0 * (4 * B + 1)
        pairs = sum(m * L + m * (m + 1) // 2 for L, m in zip(lens, n))
        return {"bytes": b, "flops": 2.0 * D * H * pairs}
    lens, kept, moves = _need(case)
    units = case["layers"] * case["kv_heads"]
    # as many of the kept lie behind the budget as of a random choice
    moved = sum(k * (L - k) / L for L, k in zip(lens, kept))
    if op == "plan":
        over = sum(L for L, k in zip(lens, kept) if L > k)
        return {"bytes": units * (8.0 * over + 8.0 * moved + 4.0 * B) + 4.0 * 5 * B, "flops": 0.0}
    return {"bytes": units * (moved * (8.0 + 8.0 * case["dim"] + 16.0) + 4.0 * B) + 4.0 * 6 * B, "flops": 0.0}


# ------------------------------------------------------------------- inputs


def _indptr(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device="cuda")


def _pages(case, tokens, g):
    """A block table whose rows hold `tokens` tokens each, on shuffled pages."""
    need = [-(-t // case["page"]) for t in tokens]
    num_pages = sum(need) * 9 // 8 + 8
    ids = torch.randperm(num_pages - 1, generator=g, device="cuda").to(torch.int32) + 1
    width = max(max(need), 1)
    k = torch.arange(width, device="cuda")
    n, first = torch.as_tensor(need, device="cuda")[:, None], torch.as_tensor(_indptr(need)[:-1], device="cuda")[:, None]
    table = torch.where(k < n, ids[(first + k).clamp_(max=num_pages - 2)], 0)
    return num_pages, table.to(torch.int32).contiguous()


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _frequencies(case):
    """Radians per token of every pair of a head, and the factor of the rotated part."""
    R, base = case["rot"], 1e6
    i = np.arange(R // 2)
    f = base ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "parts":  # slow pairs stretched, fast ones as they were, a ramp between
        factor, length = 4.0, 32768.0
        at = [R * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _turns(f):
    """Frequencies as the library takes them: turns per token in units of 2^-64."""
    whole = [int(round(math.ldexp(x / (2 * math.pi), 64))) & (2 ** 64 - 1) for x in f]
    return torch.as_tensor(np.array(whole, dtype=np.uint64).view(np.int64), device="cuda")


def _seen_pairs(L, n):
    """[query, key] of a row: whether the query sees the key."""
    return torch.arange(L + n, device="cuda") <= L + torch.arange(n, device="cuda")[:, None]


def _log_sums(s):
    """What the attention of the step has given: log-sum-exps of the scores, row by row."""
    c, lse = s["case"], torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    K, D, G = c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    first = _indptr(_counts(c))
    for b, L in enumerate(_lens(c)):
        lo, hi = int(first[b]), int(first[b + 1])
        n = hi - lo
        k = s["k"][s["table"][b, : -(-(L + n) // c["page"])].long()]
        k = (k if c["layout"] == "nhd" else k.transpose(1, 2)).reshape(-1, K, D)[: L + n]
        q = s["q"][lo:hi].view(n, K, G, D)
        if n == 1:
            a = torch.einsum("kgd,tkd->kgt", q[0].float(), k.float()) * s["scale"]
            lse[lo] = torch.logsumexp(a, 2).view(-1)
            continue
        for h in range(K):
            a = (q[:, h].reshape(n * G, D).float() @ k[:, h].float().T).view(n, G, -1) * s["scale"]
            a = a.masked_fill_(~_seen_pairs(L, n)[:, None], -math.inf)
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(a, 2)
    return lse


def _scores(case, lens, gone, slots, g):
    """Scores and positions of a cache that has been evicted from before: the
    newest tokens in order at the end, the rest anywhere."""
    shape = (case["layers"], case["batch"], case["kv_heads"], slots)
    mass = torch.randn(shape, generator=g, device="cuda").mul_(1.5).exp_()
    s = torch.arange(slots, device="cuda")
    L, e = (torch.as_tensor(x, device="cuda")[:, None, None] for x in (lens, gone))
    new = (L // 32).clamp(min=1)
    old = (torch.rand(shape, generator=g, device="cuda") * (L + e - new)).long()
    pos = torch.where(s >= L - new, s + e, torch.where(s < case["sink"], s, old))
    return mass, pos.int().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, B = case["op"], case["batch"]
    s = {"case": case, "op": op}
    lens = _lens(case)
    s["seqlens"] = _i32(lens)
    K = case["kv_heads"]
    if op in ("plan", "apply"):
        _, kept, moves = _need(case)
        r = random.Random(case["len_seed"] + 5)
        gone = [r.randint(0, 4096) for _ in lens]
        s["gone"], s["slots"] = _i32(gone), case["len_hi"]
        s["mass"], s["pos"] = _scores(case, lens, gone, s["slots"], g)
        s["budgets"] = _i32([case["budget"]] * B)
        s["sink"], s["recent"] = case["sink"], case["recent"]
        shape = (case["layers"], B, K)
        s["moves"] = torch.full(shape + (max(1, max(moves)), 2), -1, dtype=torch.int32, device="cuda")
        s["num_moves"] = torch.zeros(shape, dtype=torch.int32, device="cuda")
        s["row_lens"] = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
        if op == "plan":
            return s
        _plain_plan(s)  # the step before: what is applied here
        pages, s["table"] = _pages(case, lens, g)
        P, D = case["page"], case["dim"]
        shape = (case["layers"], pages) + ((P, K, D) if case["layout"] == "nhd" else (K, P, D))
        s["k"], s["v"] = _normal(shape, g), _normal(shape, g)
        return s
    counts = _counts(case)
    T, H, D, P = sum(counts), case["heads"], case["dim"], case["page"]
    s["indptr"] = _i32(_indptr(counts))
    s["q"] = _normal((T, H, D), g)
    r = random.Random(case["len_seed"] + 5)
    s["gone"] = _i32([r.randint(0, case.get("gone", 4096)) for _ in lens])
    if op == "rope":
        f, s["factor"] = _frequencies(case)
        s["radians"], s["freqs"] = torch.as_tensor(f, device="cuda"), _turns(f)
        s["k_new"] = _normal((T, K, D), g)
        s["q_out"] = torch.empty_like(s["q"])
        if not case["append"]:
            row, i = _rows_of(s["indptr"], T)
            s["positions"] = (s["seqlens"][row] + s["gone"][row] + i).int()
            s["k_out"] = torch.empty_like(s["k_new"])
            return s
        s["v_new"] = _normal((T, K, D), g)
    pages, s["table"] = _pages(case, [L + n for L, n in zip(lens, counts)], g)
    shape = (pages, P, K, D) if case["layout"] == "nhd" else (pages, K, P, D)
    s["k"] = _normal(shape, g)
    if op == "rope":
        s["v"] = _normal(shape, g)
        return s
    s["scale"] = 1.0 / math.sqrt(D)
    s["count_max"], s["keys_max"] = max(counts), max(L + n for L, n in zip(lens, counts))
    s["q"].mul_(2.0)  # attention that prefers some tokens
    s["lse"] = _log_sums(s)
    s["slots"] = s["keys_max"]
    # a few steps' worth of scores are there already
    s["mass"] = torch.rand(B, K, s["slots"], generator=g, device="cuda") * (8.0 * H * s["count_max"] / (K * s["keys_max"]))
    s["pos"] = torch.zeros(B, K, s["slots"], dtype=torch.int32, device="cuda")
    s["fresh"] = None if case["fresh"] == "new" else torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------- one pass


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _rows_of(indptr, T):
    """Row and index within the row of every token."""
    t = torch.arange(T, device="cuda")
    row = torch.searchsorted(indptr[1:].long(), t, right=True).clamp_(max=indptr.numel() - 2)
    return row, t - indptr.long()[row]


def _rotate(x, cos, sin, pairing):
    """x [T, heads, D] by the angles [T, 1, R / 2] of its first R values; in 32 bits."""
    R = 2 * cos.shape[2]
    x = x.float()
    if pairing == "half":
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1).to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    row, i = _rows_of(s["indptr"], s["q"].shape[0])
    at = s["seqlens"].long()[row] + i
    pos = at + s["gone"][row] if c["append"] else s["positions"]
    angle = pos.double()[:, None] * s["radians"]  # far positions: 32 bits would lose the angle
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["pairing"]))
    k = _rotate(s["k_new"], cos, sin, c["pairing"])
    if not c["append"]:
        s["k_out"].copy_(k)
        return {"q": s["q_out"], "k": s["k_out"]}
    kc, vc = (x if c["layout"] == "nhd" else x.transpose(1, 2) for x in (s["k"], s["v"]))
    page, P = s["table"].long()[row, at // c["page"]], c["page"]
    kc[page, at % P] = k
    vc[page, at % P] = s["v_new"]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _own_rope(s):
    pkv = _lib()
    c = s["case"]
    pairing = pkv.ROPE_HALF if c["pairing"] == "half" else pkv.ROPE_INTERLEAVED
    if not c["append"]:
        pkv.pkv_rope(s["q"], s["k_new"], s["positions"], s["freqs"], pairing=pairing, attn_factor=s["factor"],
                     q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    pkv.pkv_rope_append(s["k"], s["v"], s["q"], s["k_new"], s["v_new"], s["table"], s["seqlens"], s["freqs"],
                        pairing=pairing, attn_factor=s["factor"], append_indptr=s["indptr"], evicted=s["gone"],
                        q_out=s["q_out"], layout=pkv.NHD if c["layout"] == "nhd" else pkv.HND)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_mass(s):
    c = s["case"]
    H, K, D, P = c["heads"], c["kv_heads"], c["dim"], c["page"]
    G, B, n, L = H // K, c["batch"], s["count_max"], s["seqlens"].long()
    kc = s["k"] if c["layout"] == "nhd" else s["k"].transpose(1, 2)
    at = torch.arange(s["keys_max"], device="cuda")
    page = s["table"].long()[:, (at // P).clamp(max=s["table"].shape[1] - 1)]
    keys = kc[page, at % P].permute(0, 2, 3, 1).float()                                      # [B, K, D, keys]
    i = torch.arange(n, device="cuda")
    count = (s["indptr"][1:] - s["indptr"][:-1]).long()[:, None]
    live = i < count
    tok = torch.where(live, s["indptr"][:-1].long()[:, None] + i, 0)
    q = s["q"][tok].float().view(B, n, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, n * G, D)
    weight = (q @ keys).mul_(s["scale"]).view(B, K, n, G, -1)
    weight.sub_(s["lse"][tok].view(B, n, K, G).permute(0, 2, 1, 3)[..., None]).exp_()
    seen = live[:, :, None] & (at <= (L[:, None] + i)[:, :, None])
    weight.masked_fill_(~seen[:, None, :, None], 0.0)
    got = weight.sum((2, 3))
    mine = (at < L[:, None] + count)[:, None]
    fresh = mine & (at >= (L if s["fresh"] is None else s["fresh"].long())[:, None])[:, None]
    mass, pos = s["mass"], s["pos"]
    mass.copy_(torch.where(mine, torch.where(fresh, 0.0, mass) + got, mass))
    pos.copy_(torch.where(fresh, (at + s["gone"].long()[:, None])[:, None], pos))
    return {"mass": mass, "pos": pos}


def _own_mass(s):
    pkv = _lib()
    c = s["case"]
    layout = pkv.NHD if c["layout"] == "nhd" else pkv.HND
    if "workspace" not in s:
        s["workspace"] = pkv.mass_workspace(c["batch"], s["q"].shape[0], s["table"].shape[1], c["heads"],
                                            pkv.cache_desc(s["k"], layout), s["q"].device)
    pkv.pkv_attn_mass(s["k"], s["q"], s["lse"], s["table"], s["seqlens"], s["scale"], s["mass"],
                      qo_indptr=None if s["count_max"] == 1 else s["indptr"], fresh_from=s["fresh"], evicted=s["gone"],
                      slot_pos=s["pos"], workspace=s["workspace"], layout=layout)
    return {"mass": s["mass"], "pos": s["pos"]}


def _plain_plan(s):
    mass, L, N = s["mass"], s["seqlens"].long(), s["slots"]
    total = L + s["gone"].long()
    keep = torch.minimum(L, s["budgets"].long())
    at = torch.arange(N, device="cuda")
    live = (at < L[:, None])[:, None]
    safe = (s["pos"] < s["sink"]) | (s["pos"] >= (total - s["recent"])[:, None, None])
    rank = torch.where(live, torch.where(safe, 2, 1), 0)
    # by score, then by class, both sorts stable: ties go to the lowest slot
    order = torch.sort(mass, dim=-1, descending=True, stable=True)[1]
    order = order.gather(-1, torch.sort(rank.expand(mass.shape).gather(-1, order), dim=-1, descending=True, stable=True)[1])
    kept = torch.empty_like(order).scatter_(-1, order, at.expand(mass.shape)) < keep[:, None, None]
    front = (at < keep[:, None])[:, None]
    hole, extra = front & ~kept, kept & ~front
    width = s["moves"].shape[3]
    spare = torch.full(mass.shape[:3] + (width + 1, 2), -1, dtype=torch.int32, device="cuda")
    spare[..., :width, :] = s["moves"]
    for side, flag in ((0, extra), (1, hole)):
        to = torch.where(flag, flag.int().cumsum(-1) - 1, width).clamp(max=width).long()
        spare[..., side].scatter_(-1, to, at.int().expand(mass.shape))
    s["moves"].copy_(spare[..., :width, :])
    s["num_moves"].copy_(hole.sum(-1))
    s["row_lens"].copy_(torch.stack([L, keep], 1))
    return {"moves": s["moves"], "num_moves": s["num_moves"], "row_lens": s["row_lens"]}


def _own_plan(s):
    _lib().pkv_evict_plan(s["mass"], s["pos"], s["seqlens"], s["gone"], s["budgets"], s["sink"], s["recent"],
                          moves=s["moves"], num_moves=s["num_moves"], row_lens=s["row_lens"])
    return {"moves": s["moves"], "num_moves": s["num_moves"], "row_lens": s["row_lens"]}


def _plain_apply(s):
    c = s["case"]
    P, nhd = c["page"], c["layout"] == "nhd"
    n = s["num_moves"]
    i = torch.arange(s["moves"].shape[3], device="cuda")
    l, b, h, j = torch.nonzero(i < n[..., None], as_tuple=True)
    src, dst = s["moves"][l, b, h, j].long().unbind(1)
    table = s["table"].long()
    for x in (s["k"], s["v"]):
        y = x if nhd else x.transpose(2, 3)
        y[l, table[b, dst // P], dst % P, h] = y[l, table[b, src // P], src % P, h]
    for x in (s["mass"], s["pos"]):
        x[l, b, h, dst] = x[l, b, h, src]
    s["gone"] += s["seqlens"] - s["row_lens"][:, 1]
    s["seqlens"].copy_(s["row_lens"][:, 1])
    return {k: s[k] for k in ("k", "v", "mass", "pos", "seqlens", "gone")}


def _own_apply(s):
    pkv = _lib()
    if "layers" not in s:
        s["layers"] = pkv.LayerCaches(list(s["k"]), list(s["v"]), pkv.NHD if s["case"]["layout"] == "nhd" else pkv.HND)
    pkv.pkv_evict_apply(s["layers"], s["moves"], s["num_moves"], s["row_lens"], s["table"], s["seqlens"], s["gone"],
                        mass=s["mass"], slot_pos=s["pos"])
    return {k: s[k] for k in ("k", "v", "mass", "pos", "seqlens", "gone")}


_plain = {"rope": _plain_rope, "mass": _plain_mass, "plan": _plain_plan, "apply": _plain_apply}
_own = {"rope": _own_rope, "mass": _own_mass, "plan": _own_plan, "apply": _own_apply}


# ------------------------------------------------------------------- 64 bits


def exact(case, seed):
    """Row by row in 64 bits; a plan holds whole numbers only."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "mass": _exact_mass, "apply": _exact_apply}[case["op"]](s)


def _places(s, b, lo, hi):
    """Pages and places in the page of a row's tokens lo .. hi - 1."""
    P = s["case"]["page"]
    t = torch.arange(lo, hi, device="cuda")
    return s["table"][b].long()[t // P], t % P


def _exact_rope(s):
    c, first = s["case"], _indptr(_counts(s["case"]))
    R, gone = c["rot"], s["gone"].tolist()
    got = {"q": s["q"].double(), "k": s["k_new"].double()}
    f = torch.as_tensor(_frequencies(c)[0], device="cuda")
    for b, L in enumerate(_lens(c)):
        rows = slice(int(first[b]), int(first[b + 1]))
        pos = torch.arange(rows.stop - rows.start, device="cuda", dtype=torch.float64) + (L + gone[b])
        turn = torch.polar(torch.full_like(pos[:, None] * f, s["factor"]), pos[:, None] * f)[:, None]
        for x in got.values():
            if c["pairing"] == "half":
                z = torch.complex(x[rows, :, : R // 2], x[rows, :, R // 2: R]) * turn
                x[rows, :, : R // 2], x[rows, :, R // 2: R] = z.real, z.imag
            else:
                z = torch.complex(x[rows, :, 0:R:2], x[rows, :, 1:R:2]) * turn
                x[rows, :, 0:R:2], x[rows, :, 1:R:2] = z.real, z.imag
    if not c["append"]:
        return got
    pools = {"k": s["k"].double(), "v": s["v"].double()}
    for name, new in (("k", got["k"]), ("v", s["v_new"].double())):
        y = pools[name] if c["layout"] == "nhd" else pools[name].transpose(1, 2)
        for b, L in enumerate(_lens(c)):
            lo, hi = int(first[b]), int(first[b + 1])
            page, place = _places(s, b, L, L + hi - lo)
            y[page, place] = new[lo:hi]
    return {"q": got["q"], "k": pools["k"], "v": pools["v"]}


def _exact_mass(s):
    c, first = s["case"], _indptr(_counts(s["case"]))
    K, G = c["kv_heads"], c["heads"] // c["kv_heads"]
    mass = s["mass"].double()
    kc = s["k"] if c["layout"] == "nhd" else s["k"].transpose(1, 2)
    for b, L in enumerate(_lens(c)):
        lo, hi = int(first[b]), int(first[b + 1])
        n = hi - lo
        page, place = _places(s, b, 0, L + n)
        mass[b, :, (L if c["fresh"] == "new" else 0): L + n] = 0.0
        seen = _seen_pairs(L, n)
        for h in range(K):
            k = kc[page, place, h].double()
            for g in range(h * G, (h + 1) * G):
                a = s["q"][lo:hi, g].double() @ k.T * s["scale"] - s["lse"][lo:hi, g].double()[:, None]
                mass[b, h, : L + n] += torch.where(seen, a.exp(), 0.0).sum(0)
    return {"mass": mass, "pos": None}


def _exact_apply(s):
    c = s["case"]
    moves, n, table = s["moves"].cpu().numpy(), s["num_moves"].cpu().numpy(), s["table"].cpu().numpy()
    l, b, h = (np.repeat(x.ravel(), n.ravel()) for x in np.indices(n.shape))
    pairs = np.concatenate([moves[x][: n[x]] for x in np.ndindex(*n.shape)])
    got = {"mass": s["mass"].double(), "pos": None, "seqlens": None, "gone": None}
    l, b, h = (torch.as_tensor(x, device="cuda") for x in (l, b, h))
    src, dst = (torch.as_tensor(pairs[:, x].astype(np.int64), device="cuda") for x in (0, 1))
    got["mass"][l, b, h, dst] = got["mass"][l, b, h, src]
    P, page = c["page"], torch.as_tensor(table.astype(np.int64), device="cuda")
    for name in ("k", "v"):
        x = s[name].double()
        y = x if c["layout"] == "nhd" else x.transpose(2, 3)
        y[l, page[b, dst // P], dst % P, h] = y[l, page[b, src // P], src % P, h]
        got[name] = x
    return got
