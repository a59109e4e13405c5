"""Rotary positions, accumulated attention weight and eviction (GPU): pkv_rope,
pkv_rope_append, pkv_attn_mass, pkv_evict_plan and pkv_evict_apply against
plain implementations, row fates, capture, and whole steps together with the
attention and pkv_table_update."""
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_append_gb300 as pkv
from paged_kv_decode_append_gb300 import workloads as wl

import evict_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=DEV)


def zero():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------- rotation


def freqs_of(rot, base=1e4):
    f, _ = pkv.rope_freqs(rot, base)
    return f, f.cpu().numpy().view(np.uint64)


def near(got, want, size):
    off = np.abs(got.double().cpu().numpy() - want)
    return (off <= ref.rotate_tol(want, size)).all()


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (64, 16, True), (128, 128, True), (128, 96, False),
                                         (256, 256, False), (256, 64, True), (128, 32, False), (256, 240, True)])
@pytest.mark.parametrize("T", [1, 37, 1300])
def test_rope(D, rot, inter, T):
    g = torch.Generator().manual_seed(D + rot + T)
    q, k = (torch.randn((T, h, D), generator=g).bfloat16() for h in (6, 2))
    pos = torch.randint(-5, 2 ** 31 - 1, (T,), generator=g).int()
    pos[0] = 2 ** 31 - 1
    f, fn = freqs_of(rot)
    qd, kd = q.to(DEV), k.to(DEV)
    pairing = pkv.ROPE_INTERLEAVED if inter else pkv.ROPE_HALF
    qo, ko = pkv.pkv_rope(qd, kd, i32(pos), f, pairing=pairing, attn_factor=1.25)
    for x, y in ((q, qo), (k, ko)):
        want, size = ref.rotate(x.double().numpy(), pos.tolist(), fn, inter, 1.25)
        assert near(y, want, size)
        assert same_bits(y[..., rot:], x[..., rot:].to(DEV))
    # in place, and each of the two alone
    q1, none = pkv.pkv_rope(qd, None, i32(pos), f, pairing=pairing, attn_factor=1.25, q_out=qd)
    assert none is None and q1 is qd and same_bits(qd, qo)
    _, k1 = pkv.pkv_rope(None, kd, i32(pos), f, pairing=pairing, attn_factor=1.25, k_out=kd)
    assert k1 is kd and same_bits(kd, ko)


def run_append(case, f, inter=False, factor=1.0, indptr=None, q=True, in_place=False, **more):
    kc, vc = case.k_cache.clone(), case.v_cache.clone()
    out = case.q.clone() if in_place else torch.full_like(case.q, 77.0)
    err = zero()
    pkv.pkv_rope_append(kc, vc, (out if in_place else case.q) if q else None, case.k_new, case.v_new, i32(case.block_table),
                        i32(case.cache_seqlens), f, pairing=int(inter), attn_factor=factor,
                        append_indptr=i32(case.qo_indptr if indptr is None else indptr), q_out=out if q else None,
                        err_flag=err, layout=case.layout, **more)
    torch.cuda.synchronize()
    return out, kc, vc, int(err.item())


def check_append(case, got, fn, pos, inter=False, factor=1.0, rows=None, turned=None):
    """Rotated queries, rotated keys and V in their slots, the rest as it was."""
    out, kc, vc, _ = got
    rows = range(case.batch) if rows is None else rows
    live = np.zeros(case.q.shape[0], bool)
    want_k, want_v = case.k_cache.clone(), case.v_cache.clone()
    for b in range(case.batch):
        L, lo, hi = int(case.cache_seqlens[b]), int(case.qo_indptr[b]), int(case.qo_indptr[b + 1])
        if L < 0 or hi <= lo:
            continue
        live[lo:hi] = True
        if b not in rows:
            continue
        at = np.arange(L, L + hi - lo)
        pages, slot = case.block_table[b, at // case.page_size], at % case.page_size
        view = kc if case.layout == wl.NHD else kc.transpose(1, 2)
        p, s = (torch.as_tensor(x.astype(np.int64), device=DEV) for x in (pages, slot))
        mine = view[p, s]
        want, size = ref.rotate(case.k_new[lo:hi].double().cpu().numpy(), pos[lo:hi], fn, inter, factor)
        assert near(mine, want, size), f"row {b}: keys"
        wl.scatter_tokens(want_k, case.layout, case.page_size, pages, slot, mine)
        wl.scatter_tokens(want_v, case.layout, case.page_size, pages, slot, case.v_new[lo:hi])
    assert same_bits(kc, want_k) and same_bits(vc, want_v)
    if out is None:
        return
    if turned is not None:
        live = turned
    want, size = ref.rotate(case.q.double().cpu().numpy(), pos, fn, inter, factor)
    assert near(out[torch.as_tensor(live)], want[live], size[live])
    assert bool((out[torch.as_tensor(~live)] == 77.0).all())


def positions(case, gone=None):
    gone = [0] * case.batch if gone is None else gone
    pos = np.zeros(case.q.shape[0], np.int64)
    for b in range(case.batch):
        lo, hi = int(case.qo_indptr[b]), int(case.qo_indptr[b + 1])
        pos[lo:hi] = int(case.cache_seqlens[b]) + int(gone[b]) + np.arange(hi - lo)
    return pos.tolist()


@pytest.mark.parametrize("D,Hq,Hkv,P,layout,rot,inter", [
    (128, 32, 8, 16, wl.NHD, 128, False), (256, 12, 6, 8, wl.HND, 64, True), (64, 4, 4, 1, wl.HND, 32, False),
    (128, 24, 8, 64, wl.NHD, 96, True), (64, 16, 1, 256, wl.NHD, 64, True)])
def test_rope_append(D, Hq, Hkv, P, layout, rot, inter):
    counts, lens = [1, 0, 33, 7, 130, 5], [0, 5, 40, -1, 15, 300]
    case = wl.mixed_step(3, counts, lens, Hq, Hkv, D, P, layout, device=DEV)
    f, fn = freqs_of(rot)
    gone = [0, 3, 100000, 5, 2 ** 30, 7]
    got = run_append(case, f, inter, 1.5, evicted=i32(gone))
    assert got[3] == 0
    check_append(case, got, fn, positions(case, gone), inter, 1.5)
    # positions of the caller's, and the slots as before
    pos = np.random.default_rng(1).integers(-3, 2 ** 20, case.q.shape[0])
    got = run_append(case, f, inter, positions=i32(pos), evicted=i32(gone))
    check_append(case, got, fn, pos.tolist(), inter)
    # no queries; queries in place
    got = run_append(case, f, inter, q=False)
    check_append(case, (None,) + got[1:], fn, positions(case), inter)
    there = run_append(case, f, inter)
    here = run_append(case, f, inter, in_place=True)
    live = torch.as_tensor(np.repeat(np.array(lens) >= 0, counts))
    assert same_bits(there[0][live], here[0][live]) and same_bits(there[1], here[1])


def test_rope_append_of_one_token_a_row():
    case = wl.mixed_step(4, [1] * 9, [0, 5, 16, -1, 31, 32, 100, 7, 8], 8, 2, 128, 16, device=DEV)
    f, fn = freqs_of(128)
    kc, vc, err, out = case.k_cache.clone(), case.v_cache.clone(), zero(), torch.full_like(case.q, 77.0)
    pkv.pkv_rope_append(kc, vc, case.q, case.k_new, case.v_new, i32(case.block_table), i32(case.cache_seqlens), f, q_out=out,
                        err_flag=err)
    check_append(case, (out, kc, vc, 0), fn, positions(case))
    assert int(err.item()) == 0


@pytest.mark.parametrize("T", [1217, 5000])
def test_rope_append_of_many_tokens(T):
    """Several tokens a CTA, rows that begin within one."""
    rng = np.random.default_rng(T)
    cuts = np.sort(rng.choice(np.arange(1, T), 40, replace=False))
    counts = np.diff(np.concatenate([[0], cuts, [T]]))
    lens = rng.integers(0, 50, 41)
    lens[7] = -1
    case = wl.mixed_step(5, counts, lens, 2, 1, 64, 16, device=DEV)
    case.block_table[3, int(lens[3]) // 16] = case.num_pages
    f, fn = freqs_of(64)
    got = run_append(case, f)
    assert got[3] == pkv.api.ERR_PAGE
    check_append(case, got, fn, positions(case), rows=[b for b in range(41) if b != 3])


def test_rope_append_row_fates():
    """Bad pages and overflow drop a row's append, not its queries; malformed
    ranges and tokens behind the last row are left alone."""
    case = wl.mixed_step(6, [3, 20, 5, 4, 6], [10, 20, 16, 3, 9], 8, 2, 64, 8, device=DEV)
    f, fn = freqs_of(64)
    for bad in (0, -3, case.num_pages, 2 ** 31 - 1):
        case.block_table[1, 4] = bad
        got = run_append(case, f)
        assert got[3] == pkv.api.ERR_PAGE
        check_append(case, got, fn, positions(case), rows=[0, 2, 3, 4])
    case.block_table[1, 4] = 0
    long = case.cache_seqlens.copy()
    case.cache_seqlens[1] = case.max_blocks * 8 - 19
    got = run_append(case, f)
    assert got[3] == pkv.api.ERR_OVERFLOW
    check_append(case, got, fn, positions(case), rows=[0, 2, 3, 4])
    case.cache_seqlens[1] = 2 ** 31 - 1
    assert run_append(case, f)[3] == pkv.api.ERR_OVERFLOW
    case.cache_seqlens[:] = long
    case = wl.mixed_step(6, [3, 20, 5, 4, 6], [10, 20, 16, 3, 9], 8, 2, 64, 8, device=DEV)
    good = case.qo_indptr.copy()
    bad = good.copy()
    bad[4] = 1000  # rows 3 and 4 malformed: [28, 1000) and [1000, 38)
    got = run_append(case, f, indptr=bad)
    live = np.arange(38) < 28
    check_append(case, got, fn, positions(case), rows=[0, 1, 2], turned=live)
    bad = good.copy()
    bad[1] = -5   # rows 0 and 1
    got = run_append(case, f, indptr=bad)
    check_append(case, got, fn, positions(case), rows=[2, 3, 4], turned=np.arange(38) >= 23)


@pytest.mark.parametrize("P,n", [(8, 2043), (8, 2044), (1, 700)])
def test_append_of_rows_of_many_pages(P, n):
    """Hundreds of pages to a row: good rows, and a bad page anywhere."""
    f, fn = freqs_of(64)
    case = wl.mixed_step(31, [n, 3], [5, 9], 4, 2, 64, P, device=DEV)
    got = run_append(case, f)
    assert got[3] == 0
    check_append(case, got, fn, positions(case))
    table = case.block_table.copy()
    for at, page in ((5 // P, 0), ((5 + n - 1) // P, -1), ((5 + n // 2) // P, case.num_pages)):
        case.block_table = table.copy()
        case.block_table[0, at] = page
        got = run_append(case, f)
        assert got[3] == pkv.api.ERR_PAGE
        check_append(case, got, fn, positions(case), rows=[1])


# ------------------------------------------------------------------- mass


def append_all(case):
    """The step's keys in their slots, as the attention has left them."""
    for b in range(case.batch):
        L, lo, hi = int(case.cache_seqlens[b]), int(case.qo_indptr[b]), int(case.qo_indptr[b + 1])
        if L >= 0 and hi > lo:
            at = np.arange(L, L + hi - lo)
            wl.scatter_tokens(case.k_cache, case.layout, case.page_size, case.block_table[b, at // case.page_size],
                              at % case.page_size, case.k_new[lo:hi])


def lse_all(case):
    z = torch.zeros(case.q.shape[:2], dtype=torch.float64)
    for b in range(case.batch):
        L, lo, hi = int(case.cache_seqlens[b]), int(case.qo_indptr[b]), int(case.qo_indptr[b + 1])
        if L >= 0 and hi > lo:
            z[lo:hi] = ref.lse_of(case, b, lo, hi - lo, L)
    return z.float()


def mass_case(seed, counts, lens, Hq, Hkv, D, P, layout=wl.NHD, sharp=2.0, **kw):
    case = wl.mixed_step(seed, counts, lens, Hq, Hkv, D, P, layout, device=DEV, **kw)
    case.q = (case.q.float() * sharp).bfloat16()
    append_all(case)
    return case, lse_all(case)


def run_mass(case, lse, slots=None, fresh=None, gone=None, pos=True, ws=None, old=None, indptr=True, **more):
    slots = old.shape[-1] if old is not None else case.max_blocks * case.page_size + 3 if slots is None else slots
    K = case.num_kv_heads
    if old is None:
        old = torch.rand((case.batch, K, slots), generator=torch.Generator().manual_seed(1))
    mass = old.to(DEV)
    where = torch.full((case.batch, K, slots), -9, dtype=torch.int32, device=DEV) if pos else None
    err = zero()
    ptr = more.pop("ptr", case.qo_indptr)
    pkv.pkv_attn_mass(case.k_cache, case.q, lse.to(DEV), i32(case.block_table), i32(case.cache_seqlens), case.softmax_scale,
                      mass, qo_indptr=i32(ptr) if indptr else None, fresh_from=None if fresh is None else i32(fresh),
                      evicted=None if gone is None else i32(gone), slot_pos=where, workspace=ws, err_flag=err,
                      layout=case.layout, **more)
    torch.cuda.synchronize()
    return old, mass.cpu(), None if where is None else where.cpu(), int(err.item())


def check_mass(case, lse, got, fresh=None, gone=None, rows=None, keys=None):
    old, mass, pos, _ = got
    want, tol = old.double().numpy().copy(), np.zeros(old.shape)
    wpos = np.full(old.shape, -9)
    for b in range(case.batch) if rows is None else rows:
        L, lo, n = int(case.cache_seqlens[b]), int(case.qo_indptr[b]), int(np.diff(case.qo_indptr)[b])
        if L < 0 or n <= 0:
            continue
        w, t = ref.mass_row(case, b, lo, n, L, lse)
        at = np.arange(L + n)
        new = at >= (L if fresh is None else int(fresh[b]))
        stay = np.zeros(L + n, bool) if keys is None else ~keys[b][: L + n]
        was = want[b, :, : L + n].copy()
        total = np.where(new, 0.0, was) + w
        want[b, :, : L + n] = np.where(stay, was, total)
        # the sum with what was there rounds once more
        tol[b, :, : L + n] = np.where(stay, 0.0, t + 2.0 ** -23 * total)
        wpos[b, :, : L + n] = np.where(new & ~stay, at + (0 if gone is None else int(gone[b])), -9)
    off = np.abs(mass.double().numpy() - want)
    assert np.isfinite(mass.numpy()).all()
    assert (off <= tol).all(), f"off by {(off - tol).max()} more than the bound"
    if pos is not None:
        assert np.array_equal(pos.numpy(), wpos)


# D, Hq, Hkv, P, layout
GEOMS = [
    (128, 32, 8, 16, wl.NHD),
    (256, 48, 6, 16, wl.HND),
    (64, 8, 8, 8, wl.NHD),       # one head per kv head
    (64, 16, 1, 32, wl.HND),     # 16 heads
    (128, 24, 8, 64, wl.NHD),    # 3 heads
    (64, 128, 1, 16, wl.NHD),    # 128 heads
    (256, 70, 1, 128, wl.NHD),   # 70 heads
    (256, 4, 4, 256, wl.HND),
]


@pytest.mark.parametrize("D,Hq,Hkv,P,layout", GEOMS)
def test_mass_of_decode_steps(D, Hq, Hkv, P, layout):
    lens = [0, 1, 15, 16, 127, 128, 129, 255, 256, 257, -1, 700, 63]
    case, lse = mass_case(11, [1] * 13, lens, Hq, Hkv, D, P, layout)
    gone = list(range(0, 1300, 100))
    check_mass(case, lse, run_mass(case, lse, gone=gone), gone=gone)
    # one query a row without an indptr, and nothing new
    got = run_mass(case, lse, indptr=False, fresh=[2 ** 31 - 1] * 13)
    check_mass(case, lse, got, fresh=[2 ** 31 - 1] * 13)


@pytest.mark.parametrize("D,Hq,Hkv,P,layout", GEOMS)
def test_mass_of_mixed_steps(D, Hq, Hkv, P, layout):
    counts, lens = [1, 5, 64, 0, 130, 33, 2, 100], [40, 0, 100, 7, 300, 31, -1, 0]
    case, lse = mass_case(12, counts, lens, Hq, Hkv, D, P, layout)
    check_mass(case, lse, run_mass(case, lse))
    fresh = [0, 0, 50, 0, 290, 10 ** 6, 0, -7]
    check_mass(case, lse, run_mass(case, lse, fresh=fresh, pos=False), fresh=fresh)


@pytest.mark.parametrize("D,Hq,Hkv,P,layout", [(128, 8, 2, 16, wl.NHD), (64, 2, 2, 8, wl.HND), (256, 8, 1, 16, wl.HND)])
def test_mass_of_prompts(D, Hq, Hkv, P, layout):
    """Rows of many query tiles: causal, ragged, with and without a prefix."""
    case, lse = mass_case(13, [700, 257, 1, 512], [0, 130, 900, 1], Hq, Hkv, D, P, layout)
    check_mass(case, lse, run_mass(case, lse))


@pytest.mark.parametrize("D,Hq,Hkv,P,layout", [(128, 8, 2, 16, wl.NHD), (64, 2, 2, 64, wl.HND), (64, 16, 1, 8, wl.NHD)])
def test_mass_of_few_queries_on_long_contexts(D, Hq, Hkv, P, layout):
    """Blocks of four key tiles, and the rows next to where they begin."""
    q = 128 // (Hq // Hkv)  # queries of a tile
    counts, lens = [2 * q + 3, q + 1, 12 * q, 12 * q + 1, 2 * q], [3 * 256 + 7, 512, 12 * 256 + 1, 13 * 256, 511]
    case, lse = mass_case(21, counts, lens, Hq, Hkv, D, P, layout)
    check_mass(case, lse, run_mass(case, lse))
    for b in (0, 2):  # alone: cut into more pieces
        case, lse = mass_case(22 + b, counts[b:b + 1], lens[b:b + 1], Hq, Hkv, D, P, layout)
        check_mass(case, lse, run_mass(case, lse))


def test_mass_is_the_weight_of_the_attention():
    """With the lse that the attention calls write: every query and head gives
    one in all (a weight is as exact as the attention's lse, 1e-3 of it here)."""
    case = wl.mixed_step(14, [1, 9, 40], [100, 0, 300], 8, 2, 128, 16, device=DEV)
    lse = torch.empty(case.q.shape[:2], dtype=torch.float32, device=DEV)
    pkv.pkv_mixed_attn(case.k_cache, case.v_cache, case.q, case.k_new, case.v_new, i32(case.qo_indptr), i32(case.block_table),
                       i32(case.cache_seqlens), case.softmax_scale, 64, lse=lse)
    _, mass, _, err = run_mass(case, lse.cpu(), fresh=[0, 0, 0], old=torch.zeros(3, 2, 400))
    assert err == 0
    for b, n in enumerate((1, 9, 40)):
        assert np.allclose(mass[b].sum(1).numpy(), 4 * n, rtol=1e-3)


def test_mass_row_fates():
    case, lse = mass_case(15, [1, 3, 40, 2, 6], [40, 20, 100, 9, 30], 8, 2, 128, 16)
    # more keys than scores have room for, or the table
    got = run_mass(case, lse, slots=100)
    assert got[3] == pkv.api.ERR_OVERFLOW
    check_mass(case, lse, got, rows=[0, 1, 3, 4])
    kept = case.cache_seqlens.copy()
    for huge in (case.max_blocks * 16 - 39, 2 ** 31 - 1):
        case.cache_seqlens[2] = huge
        got = run_mass(case, lse, slots=case.max_blocks * 16 + 64)
        assert got[3] == pkv.api.ERR_OVERFLOW
        check_mass(case, lse, got, rows=[0, 1, 3, 4])
    case.cache_seqlens[:] = kept
    # ranges
    for i, v in ((2, 1000), (2, -1)):
        ptr = case.qo_indptr.copy()
        ptr[i] = v  # rows 1 and 2
        got = run_mass(case, lse, ptr=ptr)
        assert got[3] == pkv.api.ERR_QLEN
        check_mass(case, lse, got, rows=[0, 3, 4])
    # slots on bad pages stay as they are
    for bad in (0, -1, case.num_pages, 2 ** 31 - 1):
        was = int(case.block_table[2, 3])
        case.block_table[2, 3] = bad
        got = run_mass(case, lse)
        case.block_table[2, 3] = was
        assert got[3] == pkv.api.ERR_PAGE
        keys = {b: np.ones(200, bool) for b in range(5)}
        keys[2][48:64] = False
        check_mass(case, lse, got, keys=keys)


def test_mass_is_not_reached_by_what_is_masked():
    """NaN and infinities in keys past the row, in other rows' queries and in
    queries that do not see a key; a query that saw nothing gives nothing."""
    case, lse = mass_case(16, [5, 3, 8], [70, 0, 120], 4, 2, 64, 8)
    clean = run_mass(case, lse)
    check_mass(case, lse, clean)
    assert torch.isnan(case.k_cache.float()).any()  # slots without a token are NaN
    # the first query of row 2 is NaN: what only later queries see stays clean
    q = case.q.clone()
    case.q[8] = NAN
    got = run_mass(case, lse)
    assert torch.isnan(got[1][2, :, :121]).all()
    assert same_bits(got[1][2, :, 121:], clean[1][2, :, 121:]) and same_bits(got[1][:2], clean[1][:2])
    case.q[8] = INF
    got = run_mass(case, lse)
    assert same_bits(got[1][2, :, 121:], clean[1][2, :, 121:]) and same_bits(got[1][:2], clean[1][:2])
    case.q.copy_(q)
    dead = lse.clone()
    dead[9] = -INF
    check_mass(case, dead, run_mass(case, dead))


def test_mass_repeats_bit_for_bit_and_shares_a_workspace():
    case, lse = mass_case(17, [600, 1, 300], [100, 900, 0], 8, 2, 128, 16)
    desc = pkv.cache_desc(case.k_cache, case.layout)
    ws = pkv.mass_workspace(case.batch, case.q.shape[0], case.max_blocks, 8, desc, DEV)
    first = run_mass(case, lse, ws=ws)
    check_mass(case, lse, first)
    small, small_lse = mass_case(18, [2, 1, 0], [3, 5, 7], 8, 2, 128, 16)
    for _ in range(3):
        check_mass(small, small_lse, run_mass(small, small_lse, ws=ws))
        assert same_bits(run_mass(case, lse, ws=ws)[1], first[1])


def test_mass_adds_up_over_steps_and_in_graphs():
    case, lse = mass_case(19, [1] * 6, [5, 60, 200, 33, 0, 128], 8, 2, 64, 8)
    slots = case.max_blocks * 8
    desc = pkv.cache_desc(case.k_cache, case.layout)
    ws = pkv.mass_workspace(6, 6, case.max_blocks, 8, desc, DEV)
    mass, z = torch.zeros(6, 2, slots, device=DEV), lse.to(DEV)
    table, lens, none = i32(case.block_table), i32(case.cache_seqlens), i32([2 ** 31 - 1] * 6)

    def step():
        pkv.pkv_attn_mass(case.k_cache, case.q, z, table, lens, case.softmax_scale, mass, fresh_from=none, workspace=ws,
                          layout=case.layout)

    step()
    torch.cuda.synchronize()
    once = mass.clone()
    mass.zero_()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
        step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, (once + once) + (once + once))


def test_mass_of_the_largest_batch():
    rng = np.random.default_rng(3)
    lens = rng.integers(-1, 40, 1024)
    case, lse = mass_case(20, [1] * 1024, lens, 2, 1, 64, 8)
    check_mass(case, lse, run_mass(case, lse))


def test_mass_of_long_rows():
    """Positions past what a work range of one CTA holds, far apart lengths."""
    case, lse = mass_case(21, [3, 1, 1], [40000, 70, 9], 4, 1, 64, 64)
    check_mass(case, lse, run_mass(case, lse))


# ------------------------------------------------------------------- plan


def plan(mass, pos, lens, gone, budgets, sink, recent, max_moves=None):
    layers, B, K, slots = mass.shape
    width = max(1, slots // 2) if max_moves is None else max_moves
    moves = torch.full((layers, B, K, width, 2), -5, dtype=torch.int32, device=DEV)
    num = torch.full((layers, B, K), -5, dtype=torch.int32, device=DEV)
    rows = torch.full((B, 2), -5, dtype=torch.int32, device=DEV)
    err = zero()
    pkv.pkv_evict_plan(torch.as_tensor(mass, device=DEV), i32(pos), i32(lens), None if gone is None else i32(gone),
                       i32(budgets), sink, recent, moves=moves, num_moves=num, row_lens=rows, err_flag=err)
    torch.cuda.synchronize()
    return moves.cpu().numpy(), num.cpu().numpy(), rows.cpu().numpy(), int(err.item())


def check_plan(mass, pos, lens, gone, budgets, sink, recent, got, failed=()):
    moves, num, rows, _ = got
    layers, B, K, slots = mass.shape
    for b in range(B):
        L, e = int(lens[b]), 0 if gone is None else int(gone[b])
        keeps = b in failed or L < 0 or budgets[b] < 0
        assert rows[b].tolist() == [L, L if keeps else min(L, int(budgets[b]))]
        for l in range(layers):
            for h in range(K):
                want = [] if keeps else ref.plan_row(mass[l, b, h], pos[l, b, h], L, e, int(budgets[b]), sink, recent)
                n = len(want)
                assert num[l, b, h] == n
                assert moves[l, b, h, :n].tolist() == [list(m) for m in want]
                assert (moves[l, b, h, n:] == -5).all()


@pytest.mark.parametrize("slots,layers,K", [(64, 3, 2), (301, 2, 3), (2112, 1, 2), (4999, 1, 1)])
def test_plan(slots, layers, K):
    rng = np.random.default_rng(slots)
    B = 9
    lens = rng.integers(1, slots + 1, B)
    lens[:4] = [slots, 0, -1, 1]
    budgets = rng.integers(0, slots, B)
    budgets[4:8] = [0, -1, 1, slots]
    budgets[0] = slots // 2
    gone = rng.integers(0, 1000, B)
    mass = np.exp(3 * rng.standard_normal((layers, B, K, slots))).astype(np.float32)
    pos = rng.integers(0, 1000 + slots, (layers, B, K, slots))
    got = plan(mass, pos, lens, gone, budgets, 4, 20)
    assert got[3] == 0
    check_plan(mass, pos, lens, gone, budgets, 4, 20, got)
    got = plan(mass, pos, lens, None, budgets, 0, 0)
    check_plan(mass, pos, lens, None, budgets, 0, 0, got)


@pytest.mark.parametrize("values", [[1.0], [0.0, -0.0], [0.0, 1.0], [NAN], [NAN, 1.0, INF, -INF, 3e38, 1e-45, -0.0, -1.0],
                                    [INF], [1.0, np.nextafter(np.float32(1), np.float32(2))]])
def test_plan_of_ties_and_special_values(values):
    rng = np.random.default_rng(7)
    slots, B = 333, 8
    mass = rng.choice(np.array(values, np.float32), (2, B, 1, slots)).astype(np.float32)
    pos = rng.integers(0, 500, (2, B, 1, slots))
    lens, budgets = [333, 333, 333, 200, 64, 33, 32, 31], [1, 332, 100, 100, 32, 32, 31, 30]
    for sink, recent in ((0, 0), (30, 40), (500, 0)):
        got = plan(mass, pos, lens, [100] * B, budgets, sink, recent)
        check_plan(mass, pos, lens, [100] * B, budgets, sink, recent, got)


@pytest.mark.parametrize("slots,budget", [(40000, 7000), (33000, 32999), (70001, 35000)])
def test_plan_of_long_rows(slots, budget):
    rng = np.random.default_rng(slots)
    mass = rng.standard_normal((1, 2, 1, slots)).astype(np.float32) ** 2
    mass[0, 1] = np.round(mass[0, 1], 1)  # many equal
    pos = np.tile(np.arange(slots), (1, 2, 1, 1))
    lens = [slots, slots - 77]
    got = plan(mass, pos, lens, None, [budget, min(budget, slots - 78)], 4, 100)
    check_plan(mass, pos, lens, None, [budget, min(budget, slots - 78)], 4, 100, got)


@pytest.mark.parametrize("slots", [128, 129, 513, 1153, 2177, 4352, 4353, 8704, 8706, 17408, 17409, 38912, 38913])
@pytest.mark.parametrize("low", [None, -1e-30, -0.0, NAN])
def test_plan_at_the_ends_of_its_variants(slots, low):
    rng = np.random.default_rng(slots)
    lens, budgets = [slots, slots - 1, slots // 2 + 1, slots], [slots // 2, 77, 60, slots - 1]
    mass = np.exp(2 * rng.standard_normal((1, 4, 1, slots))).astype(np.float32)
    if low is not None:
        mass[0, :, 0, rng.integers(0, slots)] = low  # rows of masses that are not all 0 .. +inf
        mass[0, 3, 0, : slots // 3] = low
        mass[0, 1, 0, -1] = np.uint32(0xffffffff).view(np.float32)
    pos = np.tile(np.arange(slots), (1, 4, 1, 1))
    check_plan(mass, pos, lens, None, budgets, 3, 40, plan(mass, pos, lens, None, budgets, 3, 40))
    # more protected slots than stay: some, all, and exactly as many
    for sink, recent in ((3, slots // 2 + 9), (slots, 0), (0, 77), (0, 60)):
        check_plan(mass, pos, lens, None, budgets, sink, recent, plan(mass, pos, lens, None, budgets, sink, recent))


def test_plan_row_fates():
    rng = np.random.default_rng(8)
    mass = rng.random((1, 4, 2, 100)).astype(np.float32)
    pos = rng.integers(0, 100, (1, 4, 2, 100))
    lens, budgets = [101, 100, 60, 2 ** 31 - 1], [50, 50, 10, -1]
    got = plan(mass, pos, lens, None, budgets, 2, 8)
    assert got[3] == pkv.api.ERR_OVERFLOW  # row 0 has more slots than there are scores; row 3 keeps all
    check_plan(mass, pos, lens, None, budgets, 2, 8, got, failed=[0])
    lens = [100, 100, 60, 20]
    got = plan(mass, pos, lens, None, budgets, 2, 8, max_moves=49)
    assert got[3] == pkv.api.ERR_OVERFLOW  # rows 0 and 1 may need 50 moves
    check_plan(mass, pos, lens, None, budgets, 2, 8, got, failed=[0, 1])


# ------------------------------------------------------------------- apply


class Caches:
    """Pools of several layers over one block table, with scores and positions."""

    def __init__(self, layers, lens, K, D, P, layout, slots=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.P, self.layout, B = np.array(lens), P, layout, len(lens)
        need = [-(-max(0, L) // P) for L in lens]
        self.num_pages, self.width = sum(need) + 4, max(1, max(need))
        order = torch.randperm(self.num_pages - 1, generator=g).numpy() + 1
        self.table = wl.assign_pages(np.array(need), self.num_pages, self.width, order.astype(np.int32))
        shape = (self.num_pages, P, K, D) if layout == wl.NHD else (self.num_pages, K, P, D)
        self.k, self.v = ([torch.randn(shape, generator=g).bfloat16().to(DEV) for _ in range(layers)] for _ in range(2))
        self.slots = max(1, max(lens)) if slots is None else slots
        self.mass = torch.rand((layers, B, K, self.slots), generator=g).to(DEV)
        self.pos = torch.randint(0, self.slots, (layers, B, K, self.slots), generator=g).int().to(DEV)
        self.gone = i32(range(5, 5 + B))

    def clone(self):
        return [[t.clone() for t in self.k], [t.clone() for t in self.v], self.mass.clone(), self.pos.clone()]

    def apply(self, moves, num, rows, table=None, lens=True, state=True):
        err, L = zero(), i32(self.lens)
        gone = self.gone.clone()
        pkv.pkv_evict_apply(pkv.LayerCaches(self.k, self.v, self.layout), moves, num, rows,
                            i32(self.table if table is None else table), L if lens else None, gone if lens else None,
                            mass=self.mass if state else None, slot_pos=self.pos if state else None, err_flag=err)
        torch.cuda.synchronize()
        return L.cpu().numpy(), gone.cpu().numpy(), int(err.item())

    def check(self, before, lists, rows=None, state=True):
        """lists[l][b][h]: the moves that were to be made."""
        k, v, mass, pos = before
        for l in range(len(self.k)):
            for b in range(len(self.lens)) if rows is None else rows:
                for h, m in enumerate(lists[l][b]):
                    m = [x for x in m]
                    for pool in (k[l], v[l]):
                        ref.move_slots(pool, self.layout, self.P, self.table[b], m, h)
                    if m and state:
                        src, dst = (torch.tensor(x, device=DEV) for x in zip(*m))
                        for x in (mass, pos):
                            x[l, b, h, dst] = x[l, b, h, src]
            assert same_bits(self.k[l], k[l]) and same_bits(self.v[l], v[l])
        assert same_bits(self.mass, mass) and same_bits(self.pos, pos)


def planned(c, budgets, sink=2, recent=5):
    lens = [int(x) for x in c.lens]
    moves, num, rows = pkv.pkv_evict_plan(c.mass, c.pos, i32(lens), c.gone, i32(budgets), sink, recent)
    m, n = moves.cpu().numpy(), num.cpu().numpy()
    lists = [[[[tuple(x) for x in m[l, b, h, : n[l, b, h]].tolist()] for h in range(m.shape[2])] for b in range(len(lens))]
             for l in range(m.shape[0])]
    return moves, num, rows, lists


@pytest.mark.parametrize("D,K,P,layout,layers", [(128, 8, 16, wl.NHD, 3), (64, 2, 1, wl.HND, 2), (256, 3, 256, wl.HND, 1),
                                                 (64, 1, 8, wl.NHD, 5)])
def test_apply(D, K, P, layout, layers):
    lens = [100, 33, 0, -1, 64, 500, 1]
    c = Caches(layers, lens, K, D, P, layout)
    moves, num, rows, lists = planned(c, [50, 32, 4, 4, 0, 130, 5])
    before = c.clone()
    L, gone, err = c.apply(moves, num, rows)
    assert err == 0 and L.tolist() == [50, 32, 0, -1, 0, 130, 1] and sum(map(len, lists[0][5])) > 0
    assert gone.tolist() == [55, 7, 7, 8, 73, 380, 11]
    c.check(before, lists)
    # carried out again, without the lengths: nothing changes
    again = c.clone()
    c.apply(moves, num, rows, lens=False)
    c.check(again, [[[[] for _ in range(K)] for _ in lens] for _ in range(layers)])
    # scores and positions left out
    c = Caches(layers, lens, K, D, P, layout)
    before = c.clone()
    c.apply(moves, num, rows, state=False)
    c.check(before, lists, state=False)


def test_apply_of_many_moves():
    """More moves of a head than one CTA's share."""
    c = Caches(1, [6000, 900], 1, 64, 16, wl.NHD)
    moves, num, rows, lists = planned(c, [3000, 450])
    assert int(num.max()) > 1000
    before = c.clone()
    assert c.apply(moves, num, rows)[0].tolist() == [3000, 450]
    c.check(before, lists)


def test_apply_row_fates():
    c = Caches(2, [100, 90, 80], 2, 64, 16, wl.NHD)
    moves, num, rows, lists = planned(c, [40, 40, 40])
    # a bad page anywhere in the row's slots: the whole row stays
    for bad in (0, -1, c.num_pages, 2 ** 31 - 1):
        table, before = c.table.copy(), c.clone()
        table[1, 5] = bad
        L, gone, err = c.apply(moves, num, rows, table=table)
        assert err == pkv.api.ERR_PAGE and L.tolist() == [40, 90, 40] and gone.tolist() == [65, 6, 47]
        c.check(before, lists, rows=[0, 2])
    # lengths that rise, and too many slots
    for row, want in (([30, 40], pkv.api.ERR_MOVE), ([2 ** 31 - 1, 40], pkv.api.ERR_OVERFLOW), ([-1, -1], 0)):
        bad, before = rows.clone(), c.clone()
        bad[1] = i32(row)
        L, gone, err = c.apply(moves, num, bad)
        assert err == want and L.tolist() == [40, 90, 40] and gone.tolist() == [65, 6, 47]
        c.check(before, lists, rows=[0, 2])
    # moves that lead elsewhere are left out, and heads with a count out of range
    src, dst = lists[1][0][1][0]
    for at in ((100, dst), (39, dst), (src, 40), (src, -1), (-7, dst), (2 ** 31 - 1, -2 ** 31)):
        bad, before = moves.clone(), c.clone()
        bad[1, 0, 1, 0] = i32(at)
        _, _, err = c.apply(bad, num, rows)
        assert err == pkv.api.ERR_MOVE
        c.check(before, [[[m[1:] if (l, b, h) == (1, 0, 1) else m for h, m in enumerate(hs)] for b, hs in enumerate(bs)]
                         for l, bs in enumerate(lists)])
    for at in ((0, 2, 1), (0, 0, 0)):
        for n in (-1, moves.shape[3] + 1, 2 ** 31 - 1):
            bad, before = num.clone(), c.clone()
            bad[at] = n
            L, _, err = c.apply(moves, bad, rows)
            assert err == pkv.api.ERR_MOVE and L.tolist() == [40, 40, 40]
            c.check(before, [[[[] if (l, b, h) == at else m for h, m in enumerate(hs)] for b, hs in enumerate(bs)]
                             for l, bs in enumerate(lists)])


# ------------------------------------------------------------------- together


@pytest.mark.parametrize("D,Hq,Hkv,P,layout", [(128, 8, 2, 16, wl.NHD), (64, 4, 4, 8, wl.HND)])
def test_decoding_inside_a_budget(D, Hq, Hkv, P, layout):
    """Prompts, then decode steps whose rows stay at a budget: rotation by the
    tokens' positions, attention, weights, plan, moves and tables on the device;
    a mirror keeps every head's tokens as lists."""
    layers, B, budget, steps = 2, 3, 24, 12
    sink, recent, slots = 2, 6, 48
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    rng = np.random.default_rng(5)
    pages, width = 200, -(-slots // P)
    pool = pkv.device_pool(pages)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    held, lens, gone = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    shape = (pages, P, Hkv, D) if layout == wl.NHD else (pages, Hkv, P, D)
    ks, vs = ([torch.full(shape, NAN, dtype=torch.bfloat16, device=DEV) for _ in range(layers)] for _ in range(2))
    caches = pkv.LayerCaches(ks, vs, layout)
    mass = torch.zeros(layers, B, Hkv, slots, device=DEV)
    pos = torch.zeros(layers, B, Hkv, slots, dtype=torch.int32, device=DEV)
    f, fn = freqs_of(D)
    err, budgets = zero(), i32([budget, budget, -1])
    desc = pkv.cache_desc(ks[0], layout)
    # mirror: [layer][row][head] -> lists of (position, K row, V row)
    mirror = [[[[] for _ in range(Hkv)] for _ in range(B)] for _ in range(layers)]
    for step in range(steps):
        counts = [5, 30, 17] if step == 0 else [1, 1, 1]
        indptr = np.concatenate([[0], np.cumsum(counts)])
        T = int(indptr[-1])
        tok = torch.empty(T, dtype=torch.int32, device=DEV)
        ptr = torch.empty(B + 1, dtype=torch.int32, device=DEV)
        pkv.pkv_table_update(pool, table, held, lens, i32(counts), P, indptr=ptr, positions=tok, err_flag=err)
        assert ptr.tolist() == indptr.tolist()
        old, seen_before = lens.cpu().numpy(), gone.cpu().numpy()
        for l in range(layers):
            q, k, v = (torch.as_tensor(rng.standard_normal((T, h, D)), dtype=torch.bfloat16, device=DEV)
                       for h in (Hq, Hkv, Hkv))
            q = q * 2
            lse = torch.empty(T, Hq, dtype=torch.float32, device=DEV)
            if l == 0:  # rotation and append in one call, attention over what is cached then
                qr = pkv.pkv_rope_append(ks[l], vs[l], q, k, v, table, lens, f, append_indptr=ptr, evicted=gone, err_flag=err,
                                         layout=layout)
                out = pkv.pkv_mixed_attn(ks[l], vs[l], qr, None, None, ptr, table, lens + i32(counts), scale, max(counts),
                                         lse=lse, err_flag=err, layout=layout)
            else:       # rotation alone, append by the attention
                at = torch.cat([torch.arange(n, device=DEV) + int(old[b] + seen_before[b]) for b, n in enumerate(counts)])
                qr, kr = pkv.pkv_rope(q, k, at.int(), f)
                out = pkv.pkv_mixed_attn(ks[l], vs[l], qr, kr, v, ptr, table, lens, scale, max(counts), lse=lse,
                                         err_flag=err, layout=layout)
            fresh = i32([0] * B) if step == 0 else None
            pkv.pkv_attn_mass(ks[l], qr, lse, table, lens, scale, mass[l], qo_indptr=None if step else ptr, fresh_from=fresh,
                              evicted=gone, slot_pos=pos[l], err_flag=err, layout=layout)
            # the mirror's attention, in 64 bits over its lists
            for b in range(B):
                lo, n = int(indptr[b]), counts[b]
                p0 = int(old[b] + seen_before[b])
                kk, _ = ref.rotate(k[lo:lo + n].double().cpu().numpy(), range(p0, p0 + n), fn, False)
                qq, _ = ref.rotate(q[lo:lo + n].double().cpu().numpy(), range(p0, p0 + n), fn, False)
                vv = v[lo:lo + n].double().cpu().numpy()
                for h in range(Hkv):
                    mine = mirror[l][b][h]
                    for i in range(n):
                        mine.append((p0 + i, kk[i, h], vv[i, h]))
                        K_, V_ = (np.array([m[x] for m in mine]) for x in (1, 2))
                        for g in range(h * G, (h + 1) * G):
                            s = K_ @ qq[i, g] * scale
                            w = np.exp(s - s.max())
                            want = w @ V_ / w.sum()
                            got = out[lo + i, g].double().cpu().numpy()
                            # rotated keys and queries round to bf16, 2^-8 each: scores are off by at most d, weights by a
                            # factor exp(2 d); the attention itself is within 1e-2
                            d = 2.0 ** -7 * scale * (np.abs(K_) @ np.abs(qq[i, g])).max()
                            tol = np.expm1(2 * d) * (w @ np.abs(V_ - want)) / w.sum() + 2.0 ** -8 * np.abs(want) + 1e-2
                            assert (np.abs(got - want) <= tol).all()
                    assert [m[0] for m in mine] == pos[l, b, h, : old[b] + n].tolist()
        lens += i32(counts)
        now = lens.cpu().numpy()
        m_host, p_host = mass.cpu().numpy(), pos.cpu().numpy()
        moves, num, rows = pkv.pkv_evict_plan(mass, pos, lens, gone, budgets, sink, recent, err_flag=err)
        pkv.pkv_evict_apply(caches, moves, num, rows, table, lens, gone, mass=mass, slot_pos=pos, err_flag=err)
        pkv.pkv_table_update(pool, table, held, lens, None, P, err_flag=err)
        for b in range(B):
            keep = min(int(now[b]), budget) if b < 2 else int(now[b])
            assert int(lens[b]) == keep and int(lens[b] + gone[b]) == int(now[b]) + int(seen_before[b])
            assert int(held[b]) == -(-keep // P)
            for l in range(layers):
                for h in range(Hkv):
                    mine = mirror[l][b][h]
                    for src, dst in ref.plan_row(m_host[l, b, h], p_host[l, b, h], int(now[b]), int(seen_before[b]),
                                                 int(budgets[b]), sink, recent):
                        mine[dst] = mine[src]
                    del mine[keep:]
                    kept = [m[0] for m in mine]
                    newest = int(now[b] + seen_before[b])
                    assert set(range(newest - min(recent, newest), newest)) <= set(kept) and {0, 1} <= set(kept)
        assert int(err.item()) == 0
    assert int(gone[1]) == 30 + steps - 1 - budget and int(gone[2]) == 0


def test_a_step_in_a_graph():
    """Weights, plan, moves and tables captured once and replayed: as eagerly."""
    def state():
        c = Caches(2, [60, 44, 70], 2, 64, 8, wl.NHD, slots=80, seed=9)
        c.mass.mul_(0)
        c.pos.copy_(torch.arange(80, dtype=torch.int32, device=DEV).expand_as(c.pos) + 5)
        return c

    g = torch.Generator().manual_seed(2)
    q = (2 * torch.randn((3, 4, 64), generator=g)).bfloat16().to(DEV)
    lse = torch.full((3, 4), 5.0, device=DEV)

    def step(c, lens, ws, table, outs):
        layer = pkv.LayerCaches(c.k, c.v, c.layout)
        for l in range(2):
            pkv.pkv_attn_mass(c.k[l], q, lse, table, lens, 0.125, c.mass[l], evicted=c.gone, slot_pos=c.pos[l], workspace=ws)
        pkv.pkv_evict_plan(c.mass, c.pos, lens, c.gone, budgets, 1, 4, moves=outs[0], num_moves=outs[1], row_lens=outs[2])
        pkv.pkv_evict_apply(layer, *outs, table, lens, c.gone, mass=c.mass, slot_pos=c.pos)

    budgets = i32([30, 44, 20])
    got = []
    for captured in (False, True):
        c = state()
        ws = pkv.mass_workspace(3, 3, c.width, 4, pkv.cache_desc(c.k[0]), DEV)
        table, lens = i32(c.table), i32(c.lens - 1)  # the step's own token is the last one
        outs = (torch.zeros(2, 3, 2, 40, 2, dtype=torch.int32, device=DEV), torch.zeros(2, 3, 2, dtype=torch.int32, device=DEV),
                torch.zeros(3, 2, dtype=torch.int32, device=DEV))
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(c, lens, ws, table, outs)
            graph.replay()
            graph.replay()
        else:
            step(c, lens, ws, table, outs)
            step(c, lens, ws, table, outs)
        torch.cuda.synchronize()
        got.append([*c.k, *c.v, c.mass, c.pos, lens, c.gone, *outs])
    assert got[0][6].tolist() == [30, 43, 20]
    assert all(same_bits(a, b) for a, b in zip(*got))


# ------------------------------------------------------------------- the calls themselves


def test_wrong_tensors_are_refused():
    case, lse = mass_case(22, [1, 1], [20, 5], 4, 2, 64, 8)
    f, _ = freqs_of(64)
    z, table, lens = lse.to(DEV), i32(case.block_table), i32(case.cache_seqlens)
    mass, pos = torch.zeros(2, 2, 40, device=DEV), torch.zeros(2, 2, 40, dtype=torch.int32, device=DEV)
    good = dict(k_cache=case.k_cache, q=case.q, lse=z, block_table=table, cache_seqlens=lens, softmax_scale=0.1, mass=mass,
                slot_pos=pos)
    pkv.pkv_attn_mass(**good)
    for name, bad in (("lse", z.double()), ("lse", z.cpu()), ("lse", z[:, :3]), ("q", case.q[:, :, :32].contiguous()),
                      ("q", case.q.transpose(0, 1)), ("mass", mass[:, :1].contiguous()), ("mass", mass[0]), ("mass", mass.half()),
                      ("slot_pos", pos[..., 1:].contiguous()), ("slot_pos", pos.long()), ("cache_seqlens", lens[:1]),
                      ("block_table", table.long()), ("k_cache", case.k_cache[0]), ("k_cache", case.k_cache.float()),
                      ("qo_indptr", i32([0, 1])), ("workspace", torch.zeros(64, device=DEV)), ("err_flag", torch.zeros(1))):
        with pytest.raises(ValueError):
            pkv.pkv_attn_mass(**{**good, name: bad})
    with pytest.raises(pkv.PkvError):
        pkv.pkv_attn_mass(**good, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        pkv.pkv_rope(case.q, case.k_new, i32([0]), f)
    with pytest.raises(ValueError):
        pkv.pkv_rope(case.q, None, i32([0, 1]), f.int())
    with pytest.raises(ValueError):
        pkv.pkv_rope(case.q, None, i32([0, 1]), f, q_out=case.q.float())
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(case.k_cache, case.v_cache, case.q, case.k_new, case.v_new[:1], table, lens, f)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(case.k_cache, case.v_cache[:1], case.q, case.k_new, case.v_new, table, lens, f)
    with pytest.raises(TypeError):
        pkv.pkv_rope_append(case.k_cache, case.v_cache, case.q, case.k_new, case.v_new, table, lens, f, attn_factor="1")
    with pytest.raises(ValueError):
        pkv.pkv_evict_plan(mass[None], pos, lens, None, lens, 0, 0)
    with pytest.raises(ValueError):
        pkv.pkv_evict_plan(mass[None], pos[None], lens, None, lens, 2 ** 31, 0)
    moves, num, rows = pkv.pkv_evict_plan(mass[None], pos[None], lens, None, i32([3, 3]), 0, 0)
    layers = pkv.LayerCaches([case.k_cache], [case.v_cache])
    for bad in (dict(mass=mass), dict(slot_pos=pos[None].float()), dict(err_flag=lens.long())):
        with pytest.raises(ValueError):
            pkv.pkv_evict_apply(layers, moves, num, rows, table, lens, None, **bad)
    with pytest.raises(ValueError):
        pkv.pkv_evict_apply(layers, moves, num[..., :1], rows, table, lens, None)


def test_calls_of_no_tokens():
    f, _ = freqs_of(64)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, _ = pkv.pkv_rope(q, None, i32([]), f)
    assert out.shape == q.shape
    mass = torch.zeros(1, 0, 2, 8, device=DEV)
    moves, num, rows = pkv.pkv_evict_plan(mass, mass.int(), i32([]), None, i32([]), 0, 0)
    assert num.shape == (1, 0, 2) and rows.shape == (0, 2)


def test_calls_on_another_stream():
    """A step on a side stream behind a long kernel there: nothing runs ahead of it."""
    case, lse = mass_case(23, [3, 1], [60, 40], 4, 2, 64, 8)
    f, _ = freqs_of(64)
    want = run_mass(case, lse)[1]
    z, table, lens, ptr = lse.to(DEV), i32(case.block_table), i32(case.cache_seqlens), i32(case.qo_indptr)
    start = torch.rand((2, 2, case.max_blocks * 8 + 3), generator=torch.Generator().manual_seed(1)).to(DEV)
    mass, q0 = torch.empty_like(start), torch.empty_like(case.q)
    q_ref, _ = pkv.pkv_rope(case.q, None, i32([5, 6, 7, 8]), f)
    pos4 = i32([5, 6, 7, 8])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.empty(1 << 28, device=DEV)
    with torch.cuda.stream(side):
        for _ in range(10):
            big.fill_(1.0)
        mass.copy_(start)
        q0.copy_(case.q)
        pkv.pkv_attn_mass(case.k_cache, q0, z, table, lens, case.softmax_scale, mass, qo_indptr=ptr)
        q1, _ = pkv.pkv_rope(q0, None, pos4, f)
    side.synchronize()
    assert same_bits(mass.cpu(), want) and same_bits(q1, q_ref)


def test_two_graphs_share_a_workspace():
    """Rows cut between many CTAs, captured twice with one workspace, replayed in turn."""
    case, lse = mass_case(24, [900, 700], [300, 0], 8, 2, 128, 16)
    want = run_mass(case, lse, fresh=[0, 0])[1]
    ws = pkv.mass_workspace(2, 1600, case.max_blocks, 8, pkv.cache_desc(case.k_cache), DEV)
    z, table, lens, ptr, none = lse.to(DEV), i32(case.block_table), i32(case.cache_seqlens), i32(case.qo_indptr), i32([0, 0])
    mass = [torch.zeros(2, 2, want.shape[-1], device=DEV) for _ in range(2)]
    graphs = []
    for m in mass:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pkv.pkv_attn_mass(case.k_cache, case.q, z, table, lens, case.softmax_scale, m, qo_indptr=ptr, fresh_from=none,
                              workspace=ws)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for m in mass:
        for b, n in enumerate((1200, 700)):
            assert same_bits(m[b, :, :n].cpu(), want[b, :, :n])


@pytest.mark.parametrize("P", [8, 64, 128, 256])
def test_mass_of_bad_pages_of_every_size(P):
    case, lse = mass_case(25, [2, 150], [600, 450], 4, 2, 64, P)
    blk = 250 // P
    case.block_table[1, blk] = case.num_pages + 7
    got = run_mass(case, lse)
    assert got[3] == pkv.api.ERR_PAGE
    case.block_table[1, blk] = 1
    keys = {b: np.ones(700, bool) for b in range(2)}
    keys[1][blk * P:(blk + 1) * P] = False
    check_mass(case, lse, got, keys=keys)


def test_plan_of_far_positions():
    """Positions and counts at the ends of 32 bits."""
    rng = np.random.default_rng(9)
    mass = rng.random((1, 4, 1, 130)).astype(np.float32)
    pos = rng.choice(np.array([-2 ** 31, -1, 0, 1, 7, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1]), (1, 4, 1, 130))
    lens, budgets = [130, 130, 130, 100], [60, 60, 60, 60]
    gone = [2 ** 31 - 131, 2 ** 31 - 1, -2 ** 31, 0]
    for sink, recent in ((0, 0), (1, 2), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1), (8, 2 ** 30)):
        got = plan(mass, pos, lens, gone, budgets, sink, recent)
        check_plan(mass, pos, lens, gone, budgets, sink, recent, got)
