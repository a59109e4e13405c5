"""Edges of the rotary and eviction calls (GPU): sizes at which parts of a kernel
have nothing to do, slices of larger tensors, large scores, and the calls next
to the attention calls they stand beside."""
import numpy as np
import pytest
import torch

import paged_kv_decode_append_gb300 as pkv

import test_evict_gpu as base

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 2), (256, 8, 2)])
def test_mass_of_rows_of_one_tile(D, Hq, Hkv):
    """One key tile and one query for each of many rows and heads: only one of the
    warps that issue MMAs has any to issue for a query tile."""
    lens = np.random.default_rng(D).integers(0, 128, 500)
    case, lse = base.mass_case(31, [1] * 500, lens, Hq, Hkv, D, 16)
    first = base.run_mass(case, lse)
    assert first[3] == 0
    base.check_mass(case, lse, first)
    ws = pkv.mass_workspace(500, 500, case.max_blocks, Hq, pkv.cache_desc(case.k_cache), DEV)
    for _ in range(50):
        again = base.run_mass(case, lse, ws=ws)
        assert again[3] == 0 and base.same_bits(again[1], first[1])


def rows_state(layers, B, K, slots, seed):
    """Scores and positions of all layers in one tensor each."""
    g = torch.Generator().manual_seed(seed)
    mass = torch.rand((layers, B, K, slots), generator=g).to(DEV)
    pos = torch.arange(slots, dtype=torch.int32, device=DEV).expand(layers, B, K, slots).contiguous()
    return mass, pos


@pytest.mark.parametrize("B,Hq,Hkv,slots", [(3, 2, 1, 2049), (1, 1, 1, 1001), (3, 6, 2, 203), (1, 2, 1, 510)])
def test_layers_of_one_state(B, Hq, Hkv, slots):
    """Layer by layer out of one state whose layers begin on 4 bytes: weights of
    each layer, plan and moves of the last ones."""
    layers = 3
    rng = np.random.default_rng(slots)
    lens = rng.integers(slots // 2, slots - 1, B)
    case, lse = base.mass_case(slots, [1] * B, lens, Hq, Hkv, 64, 16)
    mass, pos = rows_state(layers, B, Hkv, slots, 3)
    start = mass.clone()
    # lse of tokens out of the middle of a larger tensor
    wide = torch.zeros(B + 3, Hq, device=DEV)
    wide[3:] = lse.to(DEV)
    assert any(mass[l].data_ptr() % 16 for l in range(layers)) and any(wide[i].data_ptr() % 16 for i in range(4))
    table, old = base.i32(case.block_table), base.i32(case.cache_seqlens)
    for l in range(layers):
        pkv.pkv_attn_mass(case.k_cache, case.q, wide[3:], table, old, case.softmax_scale, mass[l], slot_pos=pos[l],
                          layout=case.layout)
        want = base.run_mass(case, lse, old=start[l].cpu())
        assert base.same_bits(mass[l].cpu(), want[1])
    c = base.Caches(layers, lens + 1, Hkv, 64, 16, base.wl.NHD, slots=slots, seed=4)
    c.mass, c.pos = mass, pos
    budgets = [int(x) // 2 for x in lens]
    width = slots // 2 | 1
    moves = torch.full((layers, B, Hkv, width, 2), -5, dtype=torch.int32, device=DEV)
    num = torch.full((layers, B, Hkv), -5, dtype=torch.int32, device=DEV)
    for part in (slice(0, 1), slice(1, layers)):
        _, _, rows = pkv.pkv_evict_plan(mass[part], pos[part], base.i32(lens + 1), c.gone, base.i32(budgets), 2, 9,
                                        moves=moves[part], num_moves=num[part])
    got = [x.cpu().numpy() for x in (moves, num, rows)] + [0]
    base.check_plan(mass.cpu().numpy(), pos.cpu().numpy(), lens + 1, c.gone.cpu().numpy(), budgets, 2, 9, got)
    lists = [[[[tuple(m) for m in got[0][l, b, h, : got[1][l, b, h]].tolist()] for h in range(Hkv)] for b in range(B)]
             for l in range(layers)]
    before, length, gone, err = c.clone(), base.i32(lens + 1), c.gone.clone(), base.zero()
    for part, last in ((slice(0, 1), False), (slice(1, layers), True)):
        pkv.pkv_evict_apply(pkv.LayerCaches(c.k[part], c.v[part], c.layout), moves[part], num[part], rows, base.i32(c.table),
                            length if last else None, gone if last else None, mass=mass[part], slot_pos=pos[part], err_flag=err)
    assert int(err.item()) == 0 and length.tolist() == budgets
    c.check(before, lists)


@pytest.mark.parametrize("budget", [-1, 50, 101, 2 ** 31 - 1])
def test_plan_of_a_row_without_scores_for_all_slots(budget):
    """Its error is the row's own, whether its budget bites or not."""
    mass, pos = (x.cpu().numpy() for x in rows_state(1, 2, 2, 100, 5))
    for lens, err in (([101, 60], pkv.api.ERR_OVERFLOW), ([2 ** 31 - 1, 60], pkv.api.ERR_OVERFLOW), ([100, 60], 0), ([-1, 60], 0)):
        got = base.plan(mass, pos, lens, None, [budget, 10], 2, 3)
        assert got[3] == err
        base.check_plan(mass, pos, lens, None, [budget, 10], 2, 3, got, failed=[0] if err else [])


@pytest.mark.parametrize("counts,lens", [([1] * 5, [0, 100, 700, 1500, 129]), ([9, 40, 300], [50, 600, 0]), ([5, 700], [3000, 9])])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 2), (128, 2, 2), (128, 8, 2), (256, 6, 1)])
def test_weights_of_large_scores(D, Hq, Hkv, counts, lens):
    """Weights are as exact for scores of 200 as for small ones.

    Queries and keys are small whole numbers, so that products and their sums are
    exact in fp32 and what is off comes from the weight alone: with d = scale q.k -
    lse, one rounding of d, one of log2(e) and one of their product (3 |d| 2^-24 of
    the weight), exp2 (2^-22).  Sums: 32 terms to a run, then no more than ten
    roundings (runs, steps, pieces, halves)."""
    case, _ = base.mass_case(D + len(counts), counts, lens, Hq, Hkv, D, 16, sharp=1.0)
    g = torch.Generator().manual_seed(D)
    whole = torch.randint(-4, 5, case.k_cache.shape, generator=g).float()
    whole[..., :8] = 4
    case.k_cache.copy_(whole.to(DEV))
    q = torch.randint(-4, 5, case.q.shape, generator=g).float()
    q[..., :8] = round(6.25 * D ** 0.5)  # 200 of every score
    case.q.copy_(q.to(DEV))
    lse = base.lse_all(case)
    assert float(lse.min()) > 150
    fresh = [0] * len(lens)
    got = base.run_mass(case, lse, fresh=fresh)
    assert got[3] == 0
    scale, G = float(np.float32(case.softmax_scale)), Hq // Hkv
    for b, L in enumerate(lens):
        lo, n = int(case.qo_indptr[b]), counts[b]
        k = base.ref.row_keys(case, b, L + n)
        seen = torch.arange(L + n) <= L + torch.arange(n)[:, None]
        want, off = torch.zeros(Hkv, L + n, dtype=torch.float64), torch.zeros(Hkv, L + n, dtype=torch.float64)
        for h in range(Hq):
            d = case.q[lo:lo + n, h].double().cpu() @ k[:, h // G].T * scale - lse[lo:lo + n, h].double()[:, None]
            w = torch.where(seen, d.exp(), 0.0)
            want[h // G] += w.sum(0)
            off[h // G] += (w * torch.expm1(2.0 ** -24 * (3 * d.abs() + 4))).sum(0)
        off += 2.0 ** -24 * (42 if n * G > 1 else 0) * want + n * G * 2.0 ** -126
        assert ((got[1][b, :, : L + n].double() - want).abs() <= off).all()
