"""Speculative decoding with trees of drafted tokens (GPU): pkv_tree_build,
pkv_tree_attn, pkv_tree_accept and pkv_tree_commit against plain
implementations, row fates, capture, and whole steps together with
pkv_table_update."""
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_append_gb300 as pkv
from paged_kv_decode_append_gb300 import workloads as wl

import tree_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
# fp32 log-sum-exp of fp32 scores: within the weights' own error (see
# tree_ref.attention; scores here stay below 2^7, so delta < 2^-9) plus
# the rounding of a value below 2^7
LSE_TOL = 2.0 ** -9


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=DEV)


def trees(case, seed=0):
    rng = np.random.default_rng(seed)
    counts = np.diff(case.qo_indptr)
    return [ref.ancestor_bits(p) for p in ref.random_parents(rng, counts)]


def run_attn(case, seen, max_nodes=None, words=None, with_new=True, caches=None, ws=None, **more):
    counts = np.diff(case.qo_indptr)
    max_nodes = max(1, int(counts.max())) if max_nodes is None else max_nodes
    words = -(-max_nodes // 32) if words is None else words
    mask = seen if isinstance(seen, np.ndarray) else ref.pack(seen, words)
    kc, vc = caches if caches is not None else (case.k_cache.clone(), case.v_cache.clone())
    out = torch.full_like(case.q, float("nan"))
    lse = torch.full(case.q.shape[:2], float("nan"), dtype=torch.float32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    indptr = more.pop("indptr", case.qo_indptr)
    pkv.pkv_tree_attn(kc, vc, case.q, case.k_new if with_new else None, case.v_new if with_new else None,
                      i32(indptr), i32(mask), i32(case.block_table), i32(case.cache_seqlens), case.softmax_scale,
                      max_nodes, out=out, lse=lse, workspace=ws, err_flag=err, layout=case.layout, **more)
    torch.cuda.synchronize()
    return out, lse, int(err.item()), kc, vc


def check(case, got, want, rows=None):
    """out within the derived bound, lse, and -inf / 0 where nothing is seen."""
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    w_out, w_lse, tol = want
    for b in range(case.batch) if rows is None else rows:
        r = slice(int(case.qo_indptr[b]), int(case.qo_indptr[b + 1]))
        assert np.isfinite(out[r]).all(), f"row {b}: not finite"
        off = np.abs(out[r] - w_out[r])
        assert (off <= tol[r]).all(), f"row {b}: off by {(off - tol[r]).max()} more than the bound"
        dead = np.isneginf(w_lse[r])
        assert np.array_equal(np.isneginf(lse[r]), dead), f"row {b}: lse"
        assert (out[r][dead] == 0).all()
        assert (np.abs(lse[r][~dead] - w_lse[r][~dead]) <= LSE_TOL).all(), f"row {b}: lse"


def check_cache(case, kc, vc, appended=True, rows=None):
    """Drafted tokens bit for bit in their slots, everything else as it was."""
    want_k, want_v = case.k_cache.clone(), case.v_cache.clone()
    if appended:
        for b in range(case.batch) if rows is None else rows:
            L, lo, hi = int(case.cache_seqlens[b]), int(case.qo_indptr[b]), int(case.qo_indptr[b + 1])
            if L < 0 or hi == lo:
                continue
            pos = np.arange(L, L + hi - lo)
            pages = case.block_table[b, pos // case.page_size]
            for pool, new in ((want_k, case.k_new), (want_v, case.v_new)):
                wl.scatter_tokens(pool, case.layout, case.page_size, pages, pos % case.page_size, new[lo:hi])
    assert torch.equal(kc.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))


# D, Hq, Hkv, P, layout
GEOMS = [
    (128, 32, 8, 16, wl.NHD),
    (128, 32, 8, 16, wl.HND),
    (256, 48, 6, 16, wl.HND),
    (64, 8, 8, 8, wl.NHD),       # one head per kv head
    (64, 16, 1, 32, wl.HND),     # 16 heads
    (128, 24, 8, 64, wl.NHD),    # 3 heads: 126 rows of a tile
    (64, 10, 2, 128, wl.HND),    # 5 heads
    (256, 6, 2, 256, wl.NHD),
    (128, 128, 1, 8, wl.NHD),    # 128 heads of one kv head: a node per tile
]


def name(g):
    return f"D{g[0]}-G{g[1] // g[2]}-P{g[3]}-{'HND' if g[4] else 'NHD'}"


# one node, chains and trees below, at and past 32 and 64 nodes; an empty row,
# an inactive one, no cached token, lengths at and around page and tile ends
NODES = [1, 5, 33, 2, 64, 0, 7, 65, 16, 3, 1]
CACHE = [300, 0, 128, 1, 127, 40, -1, 700, 255, 63, 0]


@pytest.mark.parametrize("geom", GEOMS, ids=name)
@pytest.mark.parametrize("with_new", [True, False], ids=["append", "cached"])
def test_attention_matches_the_formula(geom, with_new):
    D, Hq, Hkv, P, layout = geom
    case = wl.mixed_step(300 + D + Hq + P, NODES, CACHE, Hq, Hkv, D, P, layout, device=DEV)
    seen = trees(case, D + P)
    want = ref.attention(case, seen)
    caches = None
    if not with_new:  # the drafted tokens are in the cache already
        kc, vc = case.k_cache.clone(), case.v_cache.clone()
        pkv.pkv_append(kc, vc, case.k_new, case.v_new, i32(case.block_table), i32(case.cache_seqlens),
                       i32(case.qo_indptr), layout=layout)
        case.k_cache, case.v_cache = kc, vc
        caches = (kc.clone(), vc.clone())
    got = run_attn(case, seen, with_new=with_new, caches=caches)
    assert got[2] == 0
    check(case, got, want)
    check_cache(case, got[3], got[4], appended=with_new)


@pytest.mark.parametrize("nodes", [1, 2, 31, 32, 128, 129, 255, 256])
def test_every_tree_size(nodes):
    case = wl.mixed_step(400 + nodes, [nodes, 1, nodes], [500, 77, 3], 8, 2, 128, 16, wl.NHD, device=DEV)
    seen = trees(case, nodes)
    got = run_attn(case, seen, words=8)
    assert got[2] == 0
    check(case, got, ref.attention(case, seen))


@pytest.mark.parametrize("geom", [(128, 32, 8, 16, wl.NHD), (256, 16, 2, 16, wl.HND), (64, 16, 4, 64, wl.NHD)], ids=name)
def test_long_rows_split_over_the_device(geom):
    """Rows long enough that their keys are shared out, next to short ones."""
    D, Hq, Hkv, P, layout = geom
    case = wl.mixed_step(500 + D, [9, 64, 1, 40, 2], [40000, 9000, 7001, 31, 0], Hq, Hkv, D, P, layout,
                         extra_pages=0, device=DEV)
    seen = trees(case, 5)
    got = run_attn(case, seen)
    assert got[2] == 0
    check(case, got, ref.attention(case, seen))


def test_one_row_alone():
    for L in (0, 1, 17, 128, 129, 2000, 33000):
        case = wl.mixed_step(600 + L, [3], [L], 8, 2, 128, 16, wl.NHD, extra_pages=0, device=DEV)
        seen = trees(case, L)
        got = run_attn(case, seen)
        assert got[2] == 0
        check(case, got, ref.attention(case, seen))


def test_the_largest_batch():
    rng = np.random.default_rng(8)
    case = wl.mixed_step(700, rng.integers(0, 4, 1024), rng.integers(-1, 40, 1024), 4, 2, 64, 8, wl.NHD, device=DEV)
    seen = trees(case, 8)
    got = run_attn(case, seen)
    assert got[2] == 0
    check(case, got, ref.attention(case, seen))


def test_any_mask_and_masks_that_leave_nothing():
    """Masks that are no tree's: without the node itself, with later nodes, all
    empty (with and without cached tokens); bits at and past n are ignored."""
    case = wl.mixed_step(33, [6, 9, 4, 40], [0, 70, 0, 200], 16, 4, 128, 16, wl.HND, device=DEV)
    rng = np.random.default_rng(3)
    seen = [rng.random((n, n)) < 0.4 for n in np.diff(case.qo_indptr)]
    seen[0][2] = False   # nothing at all: no cached token either
    seen[1][5] = False   # the cached tokens only
    seen[2][:] = False
    mask = ref.pack(seen, 2)
    first = 0
    for n in np.diff(case.qo_indptr):  # garbage behind the row's nodes
        wide = np.unpackbits(mask[first:first + n].view(np.uint8).reshape(n, -1), axis=1, bitorder="little")
        wide[:, n:] = 1
        mask[first:first + n] = np.packbits(wide, axis=1, bitorder="little").view(np.int32).reshape(n, -1)
        first += n
    got = run_attn(case, mask, max_nodes=40)
    assert got[2] == 0
    want = ref.attention(case, seen)
    assert np.isneginf(want[1][2]).all() and np.isneginf(want[1][15:19]).all()
    check(case, got, want)


@pytest.mark.parametrize("geom", [(128, 16, 4, 16, wl.NHD), (64, 8, 8, 32, wl.HND), (256, 8, 2, 8, wl.NHD)], ids=name)
@pytest.mark.parametrize("L", [0, 100, 250, 5000])
def test_infinities_and_nan_in_masked_places(geom, L):
    """A drafted token that only some nodes see, or none (padding), may hold
    anything: it reaches only the nodes that see it."""
    D, Hq, Hkv, P, layout = geom
    n = 20
    case = wl.mixed_step(800 + L, [n, 3], [L, 10], Hq, Hkv, D, P, layout, device=DEV)
    seen = trees(case, 4)
    seen[0][:, 15:] = False      # nodes 15 .. 19 are padding: seen by nobody
    seen[0][:, 7] = False
    seen[0][[7, 9], 7] = True    # node 7: seen by 7 and 9 alone
    case.k_new[15:17] = float("nan")
    case.k_new[17] = float("inf")
    case.v_new[15] = float("nan")
    case.v_new[16] = float("-inf")
    case.v_new[18:20] = float("inf")
    case.v_new[7, :, 3] = float("inf")
    case.v_new[7, :, 5] = float("nan")
    case.v_new[7, :, D - 1] = float("-inf")
    got = run_attn(case, seen)
    assert got[2] == 0
    want = ref.attention(case, seen)
    out = got[0].double().cpu().numpy()
    for i in (7, 9):
        assert np.isposinf(out[i, :, 3]).all() and np.isnan(out[i, :, 5]).all() and np.isneginf(out[i, :, D - 1]).all()
    got[0][[7, 9]] = 0
    for w in (want[0], want[2]):
        w[[7, 9]] = 0
    check(case, got, want)


def place(case, pool, b, pos, head):
    """The head_dim values of row b's cached position pos."""
    page, slot = int(case.block_table[b, pos // case.page_size]), pos % case.page_size
    return pool[page, slot, head] if case.layout == wl.NHD else pool[page, head, slot]


def check_kinds(case, got, want):
    """Infinities and NaN of out where the formula has them, the rest within the bound."""
    out = got[0].double().cpu().numpy()
    for kind in (np.isposinf, np.isneginf, np.isnan):
        assert np.array_equal(kind(out), kind(want[0])), kind.__name__
    fine = np.isfinite(want[0])
    assert (np.abs(out[fine] - want[0][fine]) <= want[2][fine]).all()


@pytest.mark.parametrize("geom", [(128, 16, 4, 16, wl.NHD), (64, 8, 8, 32, wl.HND), (256, 8, 2, 8, wl.NHD)], ids=name)
@pytest.mark.parametrize("L,far", [(40, 1), (300, 1), (5000, 1), (5000, 64)])
def test_infinities_and_nan_of_cached_values(geom, L, far):
    """A cached value that is not finite reaches every node of its kv head, in its
    column alone, as it does while it is drafted; whole units and split ones, and
    (far) where its weight is nothing in 32 bits."""
    D, Hq, Hkv, P, layout = geom
    case = wl.mixed_step(900 + L, [20, 3, 5], [L, 10, 77], Hq, Hkv, D, P, layout, device=DEV)
    case.q.mul_(far)  # scores within +-300: a weight is positive in 64 bits
    seen = trees(case, 11)
    seen[0][:, 7] = False
    seen[0][[7, 9], 7] = True
    inf = float("inf")
    for pos, head, col, x in [(L // 2, 0, 3, inf), (L // 3, 0, 5, float("nan")), (0, 0, D - 1, -inf), (1, 0, 8, inf),
                              (L - 1, 0, 8, -inf), (L - 1, Hkv - 1, 0, inf), (L - 2, Hkv - 1, 0, inf)]:
        place(case, case.v_cache, 0, pos, head)[col] = x
    place(case, case.v_cache, 2, 64, Hkv - 1)[:] = -inf
    case.v_new[7, 0, 3] = -inf     # against the cached infinity of that column: NaN at the two nodes that see it
    case.v_new[7, 0, 17] = inf
    got = run_attn(case, seen)
    assert got[2] == 0
    want = ref.attention(case, seen)
    check_kinds(case, got, want)
    out = got[0]
    G = Hq // Hkv
    assert torch.isposinf(out[[0, 19], :G, 3]).all() and torch.isnan(out[[7, 9], :G, 3]).all()
    assert torch.isnan(out[:20, :G, 5]).all() and torch.isnan(out[:20, :G, 8]).all()
    assert torch.isneginf(out[:20, :G, D - 1]).all() and torch.isneginf(out[23:, -G:]).all()
    assert torch.isposinf(out[:20, -G:, 0]).all() and torch.isfinite(out[20:23]).all()


def test_infinities_of_a_very_long_row():
    """Slices of millions of keys (on shared pages) whose values are all infinite:
    reading them again takes longer than a wait in the kernel may."""
    P, D, B = 256, 256, 152
    case = wl.mixed_step(1500, [1] * B, [P] * B, 1, 1, D, P, wl.NHD, device=DEV)
    blocks = 2 ** 22 // P
    table = np.tile(case.block_table[:, :1], (1, blocks + 1)).astype(np.int32)
    table[:, blocks] = case.block_table[:, 1]
    case.v_cache.fill_(float("inf"))
    case.v_cache[..., D // 2:] = float("-inf")
    case.v_new.zero_()
    kc, vc = case.k_cache.clone(), case.v_cache.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.zeros(B, 1, device=DEV)
    out = pkv.pkv_tree_attn(kc, vc, case.q, case.k_new, case.v_new, i32(case.qo_indptr), i32(np.ones((B, 1))), i32(table),
                            i32(np.full(B, 2 ** 22)), case.softmax_scale, 1, lse=lse, err_flag=err)
    assert int(err.item()) == 0
    assert torch.isposinf(out[:, 0, : D // 2]).all() and torch.isneginf(out[:, 0, D // 2:]).all()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("L", [40, 9000, 30000])
def test_nan_scores_stay_nan(L):
    """A node whose scores are NaN, all of them or those of a long run of keys,
    is NaN; its neighbours are not touched."""
    case = wl.mixed_step(1000 + L, [6, 4], [L, 50], 8, 2, 128, 16, wl.NHD, extra_pages=0, device=DEV)
    seen = trees(case, 12)
    want = ref.attention(case, seen)
    case.q[2] = float("nan")
    case.q[7, 1] = float("nan")
    got = run_attn(case, seen)
    assert got[2] == 0
    assert torch.isnan(got[0][2]).all() and torch.isnan(got[1][2]).all()
    assert torch.isnan(got[0][7, 1]).all() and torch.isnan(got[1][7, 1])
    for w in want:
        w[2] = 0
        w[7, 1] = 0
    for g in got[:2]:
        g[2] = 0
        g[7, 1] = 0
    check(case, got, want)
    # all but the last cached keys of kv head 1: every node's heads 4 .. 7
    case = wl.mixed_step(1000 + L, [6, 4], [L, 50], 8, 2, 128, 16, wl.NHD, extra_pages=0, device=DEV)
    last = (L - 1) // 16
    case.k_cache[torch.as_tensor(case.block_table[0, :last].astype(np.int64), device=DEV), :, 1] = float("nan")
    want = ref.attention(case, seen, rows=[1])
    got = run_attn(case, seen)
    assert torch.isnan(got[0][:6, 4:]).all() and torch.isnan(got[1][:6, 4:]).all()
    assert torch.isfinite(got[0][:6, :4]).all() and torch.isfinite(got[1][:6, :4]).all()
    check(case, got, want, rows=[1])


@pytest.mark.parametrize("geom", [(128, 16, 4, 16, wl.NHD), (256, 4, 2, 8, wl.HND)], ids=name)
def test_many_values_that_are_not_finite(geom):
    """Of 200 drafted tokens a third hold infinities or NaN, each seen by a few nodes."""
    D, Hq, Hkv, P, layout = geom
    case = wl.mixed_step(1300, [200, 30], [333, 10], Hq, Hkv, D, P, layout, device=DEV)
    seen = trees(case, 15)
    rng = np.random.default_rng(15)
    for j in range(0, 200, 3):
        seen[0][:, j] = False
        seen[0][rng.integers(0, 200, 2), j] = True
        x = (float("inf"), float("-inf"), float("nan"))[j // 3 % 3]
        case.v_new[j, rng.integers(0, Hkv), rng.integers(0, D, 5)] = x
    got = run_attn(case, seen, max_nodes=256)
    assert got[2] == 0
    check_kinds(case, got, ref.attention(case, seen))


def test_padding_that_is_not_finite_costs_little():
    """Nodes that nobody sees may hold anything in K and V: the call takes about
    as long as with zeros there.  (Looking every key through again for every
    column took several hundred times as long.)"""
    case = wl.mixed_step(1400, [256] * 4, [100] * 4, 16, 2, 256, 16, wl.NHD, device=DEV)
    seen = trees(case, 16)
    for s in seen:
        s[:, 200:] = False
    mask, args = i32(ref.pack(seen, 8)), (i32(case.qo_indptr), i32(case.block_table), i32(case.cache_seqlens))
    kc, vc, out = case.k_cache.clone(), case.v_cache.clone(), torch.empty_like(case.q)
    ws = pkv.tree_workspace(4, 1024, case.max_blocks, 16, 256, pkv.cache_desc(kc), DEV)

    def best(v_new):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            for _ in range(4):
                pkv.pkv_tree_attn(kc, vc, case.q, case.k_new, v_new, args[0], mask, args[1], args[2],
                                  case.softmax_scale, 256, out=out, workspace=ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    padding = torch.arange(1024, device=DEV) % 256 >= 200
    zeros, junk = case.v_new.clone(), case.v_new.clone()
    zeros[padding] = 0
    junk[padding] = float("nan")
    plain = best(zeros)
    first = out.clone()
    assert best(junk) < 4 * plain
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))


def test_values_of_the_types_ends():
    """Scores of thousands, and the lowest finite value among the values."""
    case = wl.mixed_step(41, [12, 5], [150, 20], 8, 2, 64, 16, wl.NHD, device=DEV)
    case.q.mul_(64)
    case.v_new[3] = torch.finfo(torch.bfloat16).min
    seen = trees(case, 6)
    seen[0][:, 3] = False
    seen[0][3, 3] = True
    got = run_attn(case, seen)
    want = ref.attention(case, seen)
    # lse: a value below 2^12 in fp32, and scores that are off by delta of tree_ref
    off = np.abs(got[1].double().cpu().numpy() - want[1])
    assert (off <= 2.0 ** -12 + 2.0 ** -3).all()
    rows = [i for i in range(17) if i != 3]
    diff = np.abs(got[0].double().cpu().numpy() - want[0])
    assert (diff[rows] <= want[2][rows]).all()
    assert np.isfinite(got[0].double().cpu().numpy()).all()


@pytest.mark.parametrize("alike", [True, False], ids=["equal", "random"])
@pytest.mark.parametrize("geom,L", [((128, 8, 2, 16, wl.NHD), 300), ((64, 8, 8, 32, wl.HND), 5000),
                                    ((256, 8, 2, 16, wl.NHD), 2000), ((128, 8, 2, 16, wl.NHD), 60000)],
                         ids=lambda x: str(x) if isinstance(x, int) else name(x))
def test_values_at_the_largest_of_the_type(geom, L, alike):
    """The mean of many values at the end of bf16 is finite, whatever the number of
    keys and however their scores rise on the way."""
    D, Hq, Hkv, P, layout = geom
    case = wl.mixed_step(1100 + L, [6, 40], [L, 200], Hq, Hkv, D, P, layout, extra_pages=0, device=DEV)
    if alike:
        case.q.zero_()
    top = torch.finfo(torch.bfloat16).max
    case.v_cache.fill_(top)
    case.v_new.fill_(top)
    case.v_cache[..., D // 2:] = -top
    case.v_new[..., D // 2:] = -top
    seen = trees(case, 13)
    got = run_attn(case, seen)
    assert got[2] == 0
    check(case, got, ref.attention(case, seen))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    case = wl.mixed_step(42, [7, 33], [260, 0], 8, 2, 128, 16, wl.NHD, device=DEV)
    case.softmax_scale = scale
    seen = trees(case, 7)
    got = run_attn(case, seen)
    out, lse, tol = ref.attention(case, seen)
    assert got[2] == 0
    assert (np.abs(got[0].double().cpu().numpy() - out) <= tol).all()
    # |score| below 2^8 at the largest scale: fp32 sums of 128 products off by delta < 2^-7
    assert (np.abs(got[1].double().cpu().numpy() - lse) <= 2.0 ** -7).all()


def test_a_chain_is_a_mixed_step():
    """A tree without branches is the causal rule of pkv_mixed_attn."""
    case = wl.mixed_step(43, [4, 2, 1, 3], [900, 33, 64, 0], 32, 8, 128, 16, wl.NHD, device=DEV)
    seen = [np.tril(np.ones((n, n), bool)) for n in np.diff(case.qo_indptr)]
    got = run_attn(case, seen)
    kc, vc = case.k_cache.clone(), case.v_cache.clone()
    out = pkv.pkv_mixed_attn(kc, vc, case.q, case.k_new, case.v_new, i32(case.qo_indptr), i32(case.block_table),
                             i32(case.cache_seqlens), case.softmax_scale, 4, 4)
    # both within their bounds of the same value
    want = ref.attention(case, seen)
    check(case, got, want)
    assert (np.abs(out.double().cpu().numpy() - want[0]) <= want[2]).all()
    assert torch.equal(got[3].view(torch.int16), kc.view(torch.int16))


def test_row_fates():
    # ok, inactive, too long, bad cached page, overflow, bad drafted page, no node, ok
    case = wl.mixed_step(44, [3, 2, 9, 4, 2, 5, 0, 2], [20, -1, 5, 90, 30, 12, 9, 300], 8, 2, 128, 16, wl.NHD, device=DEV)
    seen = trees(case, 9)
    want = ref.attention(case, seen, rows=[0, 7])
    table = case.block_table.copy()
    case.block_table[3, 1] = 0
    case.block_table[5, 1] = case.num_pages + 3
    case.cache_seqlens[4] = case.max_blocks * 16 - 1
    got = run_attn(case, seen, max_nodes=8)
    assert got[2] == pkv.api.ERR_PAGE | pkv.api.ERR_OVERFLOW | pkv.api.ERR_QLEN
    check(case, got, want, rows=[0, 7])
    for b in (1, 2, 3, 4, 5):
        r = slice(int(case.qo_indptr[b]), int(case.qo_indptr[b + 1]))
        assert (got[0][r] == 0).all() and torch.isneginf(got[1][r]).all(), b
    case.block_table = table
    # row 3's bad page holds cached tokens only: its drafted tokens are appended
    check_cache(case, got[3], got[4], rows=[0, 3, 7])


def test_ranges_that_leave_the_batch():
    case = wl.mixed_step(45, [3, 2, 4], [20, 7, 5], 8, 2, 64, 16, wl.NHD, device=DEV)
    seen = trees(case, 1)
    want = ref.attention(case, seen, rows=[0])
    for indptr in ([0, 3, 5, 10], [0, 3, -1, 4], [0, 3, 3, 1]):
        got = run_attn(case, seen, indptr=np.array(indptr))
        assert got[2] == pkv.api.ERR_QLEN, indptr
        if indptr[1] == 3:
            check(case, got, want, rows=[0])


@pytest.mark.parametrize("geom", [(64, 8, 2, 16, wl.NHD), (128, 8, 8, 8, wl.HND)], ids=name)
@pytest.mark.parametrize("counts,indptr", [
    ([3, 0, 0, 2], [0, 3, -1, 3, 5]),
    ([3, 0, 0, 2], [0, 3, 99, 3, 5]),
    ([2, 0, 0, 2, 0, 0, 1], [0, 2, -5, 2, 4, 77, 4, 5]),
    ([0, 0, 4, 0, 0, 0], [9, -3, 0, 4, 3, 2, 2 ** 31 - 1]),
    ([0, 0, 250, 0, 0, 0], [9, -3, 0, 250, 3, 2, 2 ** 31 - 1]),
    ([0, 0, 0, 1, 1], [-7, 2, 2, 0, 1, 2]),
])
def test_rows_among_malformed_ranges_are_served(geom, counts, indptr):
    """Rows with a range of their own are appended and attended wherever the
    malformed ones stand (their tokens cannot be found by bisection)."""
    D, Hq, Hkv, P, layout = geom
    lens = [20, 7, 33, 5, 60, 1, 90][: len(counts)]
    case = wl.mixed_step(1200, counts, lens, Hq, Hkv, D, P, layout, device=DEV)
    good = [b for b, n in enumerate(counts) if 0 < n <= 256]
    seen = trees(case, 14)
    want = ref.attention(case, seen, rows=good)
    got = run_attn(case, seen, max_nodes=256, indptr=np.array(indptr))
    assert got[2] == pkv.api.ERR_QLEN
    check(case, got, want, rows=good)
    check_cache(case, got[3], got[4], rows=good)


def test_tokens_behind_the_last_row_are_left_alone():
    case = wl.mixed_step(46, [3, 2, 4], [20, 7, 5], 8, 2, 64, 16, wl.NHD, device=DEV)
    seen = trees(case, 1)
    got = run_attn(case, seen, indptr=np.array([0, 3, 5, 5]))
    assert got[2] == 0
    assert torch.isnan(got[0][5:]).all() and torch.isnan(got[1][5:]).all()
    check(case, got, ref.attention(case, seen), rows=[0, 1])
    case.cache_seqlens[2] = -1  # nothing of the third row is appended
    check_cache(case, got[3], got[4])


def test_the_same_call_gives_the_same_bits_whatever_the_workspace_held():
    case = wl.mixed_step(47, [16, 64, 5], [9000, 800, 20000], 32, 8, 128, 16, wl.NHD, extra_pages=0, device=DEV)
    seen = trees(case, 2)
    n = pkv.pkv_tree_workspace_size(3, case.q.shape[0], case.max_blocks, 32, 64, pkv.cache_desc(case.k_cache))
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        got = run_attn(case, seen, ws=ws)
        assert got[2] == 0
        if first is None:
            first = got
        assert torch.equal(got[0].view(torch.int16), first[0].view(torch.int16))
        assert torch.equal(got[1], first[1])


def test_captured_and_replayed_on_other_lengths():
    """One captured call serves later steps: other lengths, trees and inputs."""
    case = wl.mixed_step(48, [8, 16, 3, 30], [700, 20, 3000, 0], 8, 2, 128, 16, wl.NHD, device=DEV)
    cases = [case, wl.mixed_step(49, [8, 16, 3, 30], [120, 64, -1, 50], 8, 2, 128, 16, wl.NHD, device=DEV)]
    width = max(c.max_blocks for c in cases)
    pages = max(c.num_pages for c in cases)
    kc = torch.zeros(pages, 16, 2, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    q, kn, vn = torch.empty_like(case.q), torch.empty_like(case.k_new), torch.empty_like(case.v_new)
    table, lens = torch.zeros(4, width, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    indptr, mask = i32(case.qo_indptr), torch.zeros(57, 1, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(57, 8, dtype=torch.float32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = pkv.tree_workspace(4, 57, width, 8, 30, pkv.cache_desc(kc), DEV)

    def call():
        pkv.pkv_tree_attn(kc, vc, q, kn, vn, indptr, mask, table, lens, case.softmax_scale, 30, out=out, lse=lse,
                          workspace=ws, err_flag=err)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        lens.fill_(-1)
        call()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for k, c in enumerate(cases + cases[:1]):
        seen = trees(c, k)
        kc[: c.num_pages], vc[: c.num_pages] = c.k_cache, c.v_cache
        q.copy_(c.q), kn.copy_(c.k_new), vn.copy_(c.v_new)
        table.zero_()
        table[:, : c.max_blocks] = i32(c.block_table)
        lens.copy_(i32(c.cache_seqlens))
        mask.copy_(i32(ref.pack(seen, 1)))
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        check(c, (out, lse), ref.attention(c, seen))


def test_two_streams_at_once():
    cases = [wl.mixed_step(50 + i, [16, 40], [2000 + 900 * i, 100], 16, 4, 128, 16, wl.NHD, device=DEV) for i in (0, 1)]
    seen = [trees(c, i) for i, c in enumerate(cases)]
    calls, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, s in zip(cases, seen):
        calls.append((c.k_cache.clone(), c.v_cache.clone(), c.q, c.k_new, c.v_new, i32(c.qo_indptr),
                      i32(ref.pack(s, 2)), i32(c.block_table), i32(c.cache_seqlens), c.softmax_scale, 40))
    outs = [[torch.empty_like(c.q) for _ in range(10)] for c in cases]
    wss = [pkv.tree_workspace(2, 56, c.max_blocks, 16, 40, pkv.cache_desc(c.k_cache), DEV) for c in cases]
    torch.cuda.synchronize()
    for k in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                pkv.pkv_tree_attn(*calls[i], out=outs[i][k], workspace=wss[i])
    torch.cuda.synchronize()
    for c, s, os in zip(cases, seen, outs):
        want = ref.attention(c, s)
        for o in os:
            assert (np.abs(o.double().cpu().numpy() - want[0]) <= want[2]).all()


def test_offsets_past_32_bits():
    """Pools of more than 2^32 elements, rows on their last pages."""
    P, H, D, pages = 128, 8, 128, 36000
    assert pages * P * H * D > 2 ** 32
    case = wl.mixed_step(51, [7, 18], [300, 129], 32, H, D, P, wl.NHD, device=DEV)
    far = pages - case.num_pages
    big = [torch.empty(pages, P, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    big[0][far:], big[1][far:] = case.k_cache, case.v_cache
    seen = trees(case, 3)
    want = ref.attention(case, seen)
    table = case.block_table.copy()
    case.block_table = np.where(table > 0, table + far, 0)
    got = run_attn(case, seen, caches=tuple(big))
    assert got[2] == 0
    check(case, got, want)
    # and the commit of a path there
    layers = pkv.LayerCaches([big[0]], [big[1]])
    lo = int(case.cache_seqlens[1])
    path = i32([[2, 5], [1, 17]])
    pkv.pkv_tree_commit(layers, path, i32([2, 2]), i32(case.block_table), i32(case.cache_seqlens))
    torch.cuda.synchronize()
    at = lambda pos: big[0][int(case.block_table[1, pos // P]), pos % P].view(torch.int16)  # noqa: E731
    new = case.k_new[7:].view(torch.int16)
    assert torch.equal(at(lo), new[1]) and torch.equal(at(lo + 1), new[17])


def test_rows_past_the_tokens_that_32_bits_count():
    """A table of more than 2^31 tokens: the row overflows, its neighbour is served."""
    P, H, D = 256, 1, 64
    case = wl.mixed_step(52, [5, 6], [30, 40], 4, H, D, P, wl.NHD, device=DEV)
    seen = trees(case, 4)
    table = np.full((2, 2 ** 23 + 1), case.block_table[0, 0], np.int32)
    table[1, :case.max_blocks] = case.block_table[1]
    case.block_table = table
    for L in (2 ** 31 - 260, 2 ** 31 - 3):
        case.cache_seqlens[0] = L
        k, v = case.k_cache.clone(), case.v_cache.clone()
        before = k[int(table[0, 0])].clone()
        call = (k, v, case.q, case.k_new, case.v_new, i32(case.qo_indptr), i32(ref.pack(seen, 1)), i32(table),
                i32(case.cache_seqlens), case.softmax_scale, 6)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        lse = torch.zeros(11, 4, device=DEV)
        out = pkv.pkv_tree_attn(*call, lse=lse, err_flag=err)
        assert int(err.item()) == pkv.api.ERR_OVERFLOW
        assert (out[:5] == 0).all() and torch.isneginf(lse[:5]).all()
        assert torch.equal(k[int(table[0, 0])].view(torch.int16), before.view(torch.int16))
        want, _, tol = ref.attention(case, seen, rows=[1])
        assert (np.abs(out[5:].double().cpu().numpy() - want[5:]) <= tol[5:]).all()


# ------------------------------------------------------------------- masks


@pytest.mark.parametrize("max_nodes,words", [(1, 1), (7, 1), (32, 1), (33, 2), (64, 4), (256, 8)])
def test_build_matches_the_walk(max_nodes, words):
    rng = np.random.default_rng(max_nodes)
    counts = rng.integers(0, max_nodes + 1, 37)
    counts[:3] = [max_nodes, max_nodes, 1]
    parents = ref.random_parents(rng, counts)
    parents[0] = np.arange(max_nodes) - 1         # the deepest tree
    parents[1] = np.full(max_nodes, -1)           # no tree at all
    lens = rng.integers(-1, 500, 37)
    lens[:2] = [5, 0]
    indptr = np.concatenate([[0], np.cumsum(counts)])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    mask, pos = pkv.pkv_tree_build(i32(np.concatenate(parents)), i32(indptr), i32(lens), max_nodes,
                                   mask=torch.full((int(indptr[-1]), words), 7, dtype=torch.int32, device=DEV), err_flag=err)
    want = [ref.ancestor_bits(p) if L >= 0 else np.zeros((len(p), len(p)), bool) for p, L in zip(parents, lens)]
    assert np.array_equal(mask.cpu().numpy(), ref.pack(want, words))
    depth = np.concatenate([L + s.sum(1) - 1 if L >= 0 else np.full(len(s), -1) for s, L in zip(want, lens)])
    assert np.array_equal(pos.cpu().numpy(), depth)
    assert int(err.item()) == 0


@pytest.mark.parametrize("max_nodes,words", [(70, 3), (64, 4), (130, 5), (3, 6), (200, 7), (256, 8), (129, 8)])
def test_build_writes_mask_rows_of_any_width_and_alignment(max_nodes, words):
    rng = np.random.default_rng(words)
    counts = rng.integers(0, max_nodes + 1, 9)
    counts[0] = max_nodes
    parents = ref.random_parents(rng, counts)
    indptr = np.concatenate([[0], np.cumsum(counts)])
    T = int(indptr[-1])
    want = ref.pack([ref.ancestor_bits(p) for p in parents], words)
    for at in (0, 1, 2, 4):
        room = torch.full((T * words + 8,), 7, dtype=torch.int32, device=DEV)
        mask = room[at:at + T * words].view(T, words)
        pkv.pkv_tree_build(i32(np.concatenate(parents)), i32(indptr), i32(np.zeros(9)), max_nodes, mask=mask)
        assert np.array_equal(mask.cpu().numpy(), want)
        assert (room[:at] == 7).all() and (room[at + T * words:] == 7).all()


def test_build_and_accept_refuse_what_is_no_tree():
    parents = [[-1, 0, 1], [-1, 1], [-2], [0], [-1, 0, 2, 0], [-1]]
    indptr = np.concatenate([[0], np.cumsum([len(p) for p in parents])])
    flat, lens = i32(np.concatenate(parents)), i32([4, 5, 6, 7, 8, 9])
    same = i32(np.zeros(len(flat)))
    for max_nodes, bits in ((4, pkv.api.ERR_TREE), (3, pkv.api.ERR_TREE | pkv.api.ERR_QLEN)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        mask, pos = pkv.pkv_tree_build(flat, i32(indptr), lens, max_nodes, err_flag=err)
        assert int(err.item()) == bits
        assert mask.flatten().tolist() == [1, 3, 7] + [0] * 8 + [1]
        assert pos.tolist() == [4, 5, 6] + [-1] * 8 + [9]
        err.zero_()
        path, length, after, seqlens = pkv.pkv_tree_accept(flat, same, same, i32(np.zeros(6)), i32(indptr), lens,
                                                           max_nodes, err_flag=err)
        assert int(err.item()) == bits
        assert length.tolist() == [3, 0, 0, 0, 0, 1] and after.tolist() == [0, -1, -1, -1, -1, 0]
        assert seqlens.tolist() == [7, 5, 6, 7, 8, 10]
        assert path[0].tolist()[:3] == [0, 1, 2] and (path[1:5] == -1).all()
    # a range that leaves the batch writes nothing for its nodes
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    mask = torch.full((12, 1), 7, dtype=torch.int32, device=DEV)
    pkv.pkv_tree_build(flat, i32([0, 3, 99, 3, 3, 3, 3]), lens, 4, mask=mask, err_flag=err)
    assert int(err.item()) == pkv.api.ERR_QLEN and mask.flatten().tolist() == [1, 3, 7] + [7] * 9


# ------------------------------------------------------------------- acceptance


@pytest.mark.parametrize("with_root", [True, False], ids=["root", "no-root"])
@pytest.mark.parametrize("max_nodes,max_path", [(1, 1), (9, 4), (40, 40), (256, 300)])
def test_accept_matches_the_walk(max_nodes, max_path, with_root):
    rng = np.random.default_rng(max_nodes)
    B = 70
    counts = rng.integers(0, max_nodes + 1, B)
    parents = ref.random_parents(rng, counts)
    parents[0] = np.arange(max_nodes) - 1
    counts[0] = max_nodes
    # few tokens, so that siblings often carry the same one
    draft = [rng.integers(0, 3, n) for n in counts]
    target = [rng.integers(0, 3, n) for n in counts]
    draft[0][:], target[0][:] = 1, 1  # accepted whole
    root = rng.integers(0, 3, B)
    root[0] = 1
    lens = rng.integers(-1, 50, B)
    lens[0] = 3
    indptr = np.concatenate([[0], np.cumsum(counts)])
    cat = lambda x: i32(np.concatenate(x))  # noqa: E731
    path, length, after, seqlens = pkv.pkv_tree_accept(
        cat(parents), cat(draft), cat(target), i32(root) if with_root else None, i32(indptr), i32(lens), max_nodes,
        path=torch.full((B, max_path), 99, dtype=torch.int32, device=DEV))
    for b in range(B):
        want, token = ref.accept(parents[b], draft[b], target[b], int(root[b]) if with_root else None, max_path)
        if lens[b] < 0:
            want, token = [], -1
        assert path[b].tolist() == want + [-1] * (max_path - len(want)), b
        assert int(length[b]) == len(want) and int(after[b]) == token and int(seqlens[b]) == lens[b] + len(want)


def test_accept_may_advance_the_lengths_in_place():
    lens = i32([4, -1, 0])
    pkv.pkv_tree_accept(i32([-1, 0, -1]), i32([5, 6, 7]), i32([6, 8, 9]), i32([5, 0, 7]), i32([0, 2, 2, 3]), lens, 2,
                        seqlens_out=lens)
    assert lens.tolist() == [6, -1, 1]


# ------------------------------------------------------------------- commit


@pytest.mark.parametrize("P,layout", [(1, wl.NHD), (8, wl.HND), (16, wl.NHD), (256, wl.HND)])
@pytest.mark.parametrize("H,D,layers", [(2, 64, 1), (3, 128, 4), (1, 256, 2)])
def test_commit_moves_the_accepted_tokens(P, layout, H, D, layers):
    rng = np.random.default_rng(P + D)
    counts, lens = [40, 1, 6, 256, 20, 9], [0, 5, 31, 100, -1, 7]
    kept = [[0, 3, 4, 39], [0], [], list(range(0, 256, 3)), [0, 1], [1, 2, 3, 4, 5, 6, 7, 8]]
    case = wl.mixed_step(60 + P, counts, lens, H, H, D, P, layout, device=DEV)
    pools = [[torch.randn(case.pool_shape(), device=DEV).to(torch.bfloat16) for _ in range(layers)] for _ in range(2)]
    before = [[t.clone() for t in side] for side in pools]
    width = max(len(k) for k in kept) + 2
    path = np.full((6, width), -1)
    for b, k in enumerate(kept):
        path[b, : len(k)] = k
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_tree_commit(pkv.LayerCaches(pools[0], pools[1], layout), i32(path), i32([len(k) for k in kept]),
                        i32(case.block_table), i32(lens), err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for side, old in zip(pools, before):
        for got, was in zip(side, old):
            want = was.clone()
            to, frm = (x if layout == wl.NHD else x.transpose(1, 2) for x in (want, was))
            for b, k in enumerate(kept):
                for i, node in enumerate(k if lens[b] >= 0 else []):
                    s, d = lens[b] + node, lens[b] + i
                    to[int(case.block_table[b, d // P]), d % P] = frm[int(case.block_table[b, s // P]), s % P]
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_commit_refuses_what_is_no_path():
    case = wl.mixed_step(61, [9] * 7, [20] * 7, 2, 2, 64, 16, wl.NHD, device=DEV)
    k, v = torch.randn(2, *case.pool_shape(), device=DEV).to(torch.bfloat16)
    was = k.clone()
    path = i32([[1, 1, -1], [2, 1, -1], [-1, 0, 1], [1, 2, 3], [0, 40, -1], [3, 5, 8], [4, 5, 6]])
    table = case.block_table.copy()
    table[5, 1] = 0
    table[6, 1] = case.num_pages
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for rows, bits in (([0], pkv.api.ERR_TREE), ([1], pkv.api.ERR_TREE), ([2], pkv.api.ERR_TREE),
                       ([3], pkv.api.ERR_TREE), ([4], pkv.api.ERR_OVERFLOW), ([5], pkv.api.ERR_PAGE),
                       ([6], pkv.api.ERR_PAGE)):
        length = [2, 2, 2, 4, 2, 3, 3]
        err.zero_()
        lens = i32([20 if b in rows else -1 for b in range(7)])
        pkv.pkv_tree_commit(pkv.LayerCaches([k], [v]), path, i32(length), i32(table), lens, err_flag=err)
        assert int(err.item()) == bits, rows
        assert torch.equal(k.view(torch.int16), was.view(torch.int16))


# ------------------------------------------------------------------- together


@pytest.mark.parametrize("P", [8, 16])
def test_whole_steps(P):
    """Several steps of a speculative decoder, as a serving loop runs them on
    the device: tables, masks, attention, acceptance, commit.  The cache of
    every row holds exactly the accepted tokens' K/V, and attention sees it."""
    rng = np.random.default_rng(P)
    B, Hq, Hkv, D, n, pages, width, layers = 5, 8, 2, 128, 12, 200, 24, 2
    caches = [[torch.full((pages, P, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(layers)]
              for _ in range(2)]
    both = pkv.LayerCaches(*caches)
    pool, plain = pkv.device_pool(pages), ref.TablePool(pages, B, width, P)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    held = torch.zeros(B, dtype=torch.int32, device=DEV)
    lens = i32([0, 0, 0, 0, -1])
    history = [[[] for _ in range(B)] for _ in range(layers)]  # accepted (k, v) of every row
    desc = pkv.cache_desc(caches[0][0])
    ws = pkv.tree_workspace(B, B * n, width, Hq, n, desc, DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for step in range(6):
        if step == 3:
            lens[1], lens[4] = -1, 0  # a request ends, another comes
            for h in history:
                h[1], h[4] = [], []
        host = lens.cpu().numpy()
        counts = np.where(host >= 0, rng.integers(1, n + 1, B), 0)
        T = int(counts.sum())
        indptr = torch.empty(B + 1, dtype=torch.int32, device=DEV)
        slots, pos = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV)
        pkv.pkv_table_update(pool, table, held, lens, i32(counts), P, indptr=indptr, slot_map=slots, positions=pos,
                             err_flag=err)
        want = plain.update(host, counts, T)
        assert np.array_equal(indptr.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[1])
        assert np.array_equal(table.cpu().numpy(), plain.table) and np.array_equal(held.cpu().numpy(), plain.held)
        parents = ref.random_parents(rng, counts)
        mask, positions = pkv.pkv_tree_build(i32(np.concatenate(parents)), indptr, lens, n)
        fresh = [torch.randn(2, T, Hkv, D, device=DEV).to(torch.bfloat16) for _ in range(layers)]
        q = torch.randn(T, Hq, D, device=DEV).to(torch.bfloat16)
        for layer in range(layers):
            out = pkv.pkv_tree_attn(caches[0][layer], caches[1][layer], q, fresh[layer][0], fresh[layer][1], indptr,
                                    mask, table, lens, 0.1, n, workspace=ws, err_flag=err)
            for b in range(B):
                lo, hi = int(want[0][b]), int(want[0][b + 1])
                if hi == lo:
                    continue
                old = history[layer][b]
                k = torch.cat(([torch.stack([x[0] for x in old])] if old else []) + [fresh[layer][0][lo:hi]]).double()
                v = torch.cat(([torch.stack([x[1] for x in old])] if old else []) + [fresh[layer][1][lo:hi]]).double()
                seen = torch.ones(hi - lo, len(k), dtype=torch.bool, device=DEV)
                seen[:, len(old):] = torch.as_tensor(ref.ancestor_bits(parents[b]), device=DEV)
                kk, vv = (x.repeat_interleave(Hq // Hkv, 1) for x in (k, v))
                s = torch.einsum("ihd,jhd->hij", q[lo:hi].double(), kk) * 0.1
                o = torch.einsum("hij,jhd->ihd", s.masked_fill(~seen, -math.inf).softmax(-1), vv)
                # rounding to bf16, and weights off by less than 2^-12 (tree_ref.attention at these sizes)
                assert ((out[lo:hi].double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -11 * vv.abs().max()).all()
        draft, target = i32(rng.integers(0, 3, T)), i32(rng.integers(0, 3, T))
        path, length, _, after = pkv.pkv_tree_accept(i32(np.concatenate(parents)), draft, target,
                                                     i32(rng.integers(0, 3, B)), indptr, lens, n, err_flag=err)
        pkv.pkv_tree_commit(both, path, length, table, lens, err_flag=err)
        for b in range(B):
            for node in path[b].tolist()[: int(length[b])]:
                for layer in range(layers):
                    history[layer][b].append(fresh[layer][:, int(want[0][b]) + node])
        lens = after
        for b in range(B):
            for p in range(max(0, int(lens[b]))):
                for layer in range(layers):
                    for side in (0, 1):
                        got = caches[side][layer][int(table[b, p // P]), p % P]
                        assert torch.equal(got.view(torch.int16), history[layer][b][p][side].view(torch.int16))
    assert int(err.item()) == 0
