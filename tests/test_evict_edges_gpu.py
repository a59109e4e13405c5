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


class Decoder:
    """A decoder's steps of one token a row inside a budget of slots, next to the
    decode attention: rotation, attention, weights in every layer, then plan, moves
    and tables.  One row is padding.  `way`: how keys get into the cache."""

    layers, B, slots, steps = 3, 5, 80, 8

    def __init__(self, way, D, Hq, Hkv, P, layout):
        self.way, self.D, self.G, self.P, self.layout, self.scale = way, D, Hq // Hkv, P, layout, D ** -0.5
        g = torch.Generator().manual_seed(D + P)
        pages, K, B = 150, Hkv, self.B
        shape = (pages, P, K, D) if layout == base.wl.NHD else (pages, K, P, D)
        self.ks, self.vs = ([torch.randn(shape, generator=g).bfloat16().to(DEV) for _ in range(self.layers)] for _ in range(2))
        self.caches = pkv.LayerCaches(self.ks, self.vs, layout)
        self.pool, self.held, self.gone = pkv.device_pool(pages), base.i32([0] * B), base.i32([0, 7, 100, 0, 3])
        self.table = torch.zeros(B, -(-self.slots // P), dtype=torch.int32, device=DEV)
        self.lens, self.one, self.err = base.i32([39, 24, 5, -1, 60]), base.i32([1] * B), base.zero()
        self.budgets = base.i32([30, 24, 24, 24, -1])
        pkv.pkv_table_update(self.pool, self.table, self.held, self.lens, None, P)
        self.mass = torch.rand((self.layers, B, K, self.slots), generator=g).to(DEV)
        self.pos = (torch.arange(self.slots, device=DEV) + self.gone[:, None, None]).int().expand(self.mass.shape).contiguous()
        self.inputs = [[torch.randn((self.layers, B, h, D), generator=g).bfloat16().to(DEV) for h in (Hq, K, K)]
                       for _ in range(self.steps)]
        self.now = [torch.empty_like(x) for x in self.inputs[0]]  # this step's q, k, v
        self.turned = [torch.empty_like(x) for x in self.now[:2]]
        self.out, self.lse = torch.empty_like(self.now[0]), torch.empty(self.layers, B, Hq, device=DEV)
        self.freqs, _ = pkv.rope_freqs(D)
        desc = pkv.cache_desc(self.ks[0], layout)
        self.ws = pkv.decode_workspace(B, self.table.shape[1], Hq, desc, DEV)
        self.mass_ws = pkv.mass_workspace(B, B, self.table.shape[1], Hq, desc, DEV)
        self.work = (torch.zeros(self.layers, B, K, self.slots // 2, 2, dtype=torch.int32, device=DEV),
                     torch.zeros(self.layers, B, K, dtype=torch.int32, device=DEV), torch.zeros(B, 2, dtype=torch.int32, device=DEV))
        if way == "step":
            self.graph = pkv.DecodeStep(self.ks, self.vs, list(self.turned[0]), list(self.turned[1]), list(self.now[2]),
                                        self.table, self.lens, self.scale, list(self.out), list(self.lse), self.ws, self.err,
                                        layout, pkv.api.DECODE_USE_PLAN | pkv.api.DECODE_OVERLAP_PROLOGUE)

    def attend(self, l, after, positions):
        q, k, v = (x[l] for x in self.now)
        if self.way == "append":  # rotated and appended, then attended with the lengths after
            pkv.pkv_rope_append(self.ks[l], self.vs[l], q, k, v, self.table, self.lens, self.freqs, evicted=self.gone,
                                q_out=self.turned[0][l], err_flag=self.err, layout=self.layout)
            pkv.pkv_decode_attn(self.ks[l], self.vs[l], self.turned[0][l], None, None, self.table, after, self.scale,
                                out=self.out[l], lse=self.lse[l], workspace=self.ws, err_flag=self.err, layout=self.layout)
            return
        pkv.pkv_rope(q, k, positions, self.freqs, q_out=self.turned[0][l], k_out=self.turned[1][l])
        if self.way == "step":
            return
        api = pkv.api
        flags = 0 if self.way == "fused" else api.DECODE_MAKE_PLAN if l == 0 else \
            api.DECODE_USE_PLAN | api.DECODE_OVERLAP_PROLOGUE | api.DECODE_EARLY_KV
        pkv.pkv_decode_attn(self.ks[l], self.vs[l], self.turned[0][l], self.turned[1][l], v, self.table, self.lens, self.scale,
                            out=self.out[l], lse=self.lse[l], workspace=self.ws, err_flag=self.err, layout=self.layout,
                            flags=flags)

    def step(self, look=None):
        pkv.pkv_table_update(self.pool, self.table, self.held, self.lens, self.one, self.P, err_flag=self.err)
        after = self.lens + (self.lens >= 0).int()
        positions = self.lens + self.gone
        for l in range(self.layers):
            self.attend(l, after, positions)
        if self.way == "step":
            self.graph.launch()
        for l in range(self.layers):
            if look is not None:
                look(self, l)
            pkv.pkv_attn_mass(self.ks[l], self.turned[0][l], self.lse[l], self.table, self.lens, self.scale, self.mass[l],
                              evicted=self.gone, slot_pos=self.pos[l], workspace=self.mass_ws, err_flag=self.err,
                              layout=self.layout)
            if look is not None:
                look(self, l, done=True)
        self.lens.copy_(after)
        pkv.pkv_evict_plan(self.mass, self.pos, self.lens, self.gone, self.budgets, 2, 5, *self.work, err_flag=self.err)
        pkv.pkv_evict_apply(self.caches, *self.work, self.table, self.lens, self.gone, mass=self.mass, slot_pos=self.pos,
                            err_flag=self.err)
        pkv.pkv_table_update(self.pool, self.table, self.held, self.lens, None, self.P, err_flag=self.err)

    def state(self):
        return [*self.ks, *self.vs, self.mass, self.pos, self.lens, self.gone, self.table, self.held, self.pool, self.out, self.lse,
                self.err]

    def run(self, how):
        for x in self.inputs:
            for to, new in zip(self.now, x):
                to.copy_(new)
            how()
        torch.cuda.synchronize()
        return [x.clone() for x in self.state()]


def look(s, l, done=False):
    """A step's attention and weights against 64 bits over what is cached."""
    from types import SimpleNamespace

    table, lens = s.table.cpu().numpy(), s.lens.tolist()
    if not done:
        s.was = s.mass[l].double().cpu()
        return
    K = s.mass.shape[2]
    for b, L in enumerate(lens):
        if L < 0:
            assert base.same_bits(s.mass[l, b].double().cpu(), s.was[b]) and not s.out[l, b].any()
            continue
        k, v = (base.ref.row_keys(SimpleNamespace(k_cache=x, block_table=table, page_size=s.P, layout=s.layout, num_kv_heads=K,
                                                  head_dim=s.D), b, L + 1) for x in (s.ks[l], s.vs[l]))
        assert torch.equal(v[L], s.now[2][l, b].double().cpu())
        if s.way != "append":
            assert torch.equal(k[L], s.turned[1][l, b].double().cpu())
        q = s.turned[0][l, b].double().cpu()
        want = s.was[b].clone()
        want[:, L] = 0.0
        for h in range(K * s.G):
            w = torch.softmax(k[:, h // s.G] @ q[h] * s.scale, 0)
            out = w @ v[:, h // s.G]
            assert ((s.out[l, b, h].double().cpu() - out).abs() <= 1e-2 + 1e-2 * out.abs()).all()  # the attention's bound
            want[h // s.G, : L + 1] += w
        # a weight is as exact as the attention's lse, 1e-3 of it here
        assert ((s.mass[l, b].double().cpu() - want).abs() <= 1e-3 * want).all()
        assert s.pos[l, b, :, L].tolist() == [L + int(s.gone[b])] * K


WAYS = ["fused", "plan", "append", "step"]
SHAPES = [(128, 8, 2, 16, base.wl.NHD), (64, 4, 4, 8, base.wl.HND), (256, 8, 1, 64, base.wl.NHD)]


@pytest.mark.parametrize("D,Hq,Hkv,P,layout", SHAPES)
@pytest.mark.parametrize("way", WAYS)
def test_steps_next_to_the_decode_attention(way, D, Hq, Hkv, P, layout):
    """With the fused append (and a plan shared by the layers, and a captured step of
    all layers), and with rotated keys appended before an attention alone."""
    s = Decoder(way, D, Hq, Hkv, P, layout)
    s.run(lambda: s.step(look))
    assert int(s.err.item()) == 0 and s.lens.tolist() == [30, 24, 13, -1, 68]
    assert s.gone.tolist() == [17, 15, 100, 0, 3] and s.held.tolist() == [-(-n // P) for n in (30, 24, 13, 0, 68)]


@pytest.mark.parametrize("D,Hq,Hkv,P,layout", SHAPES)
@pytest.mark.parametrize("way", WAYS[:3])
def test_whole_steps_in_a_graph(way, D, Hq, Hkv, P, layout):
    """Tables, rotation, attention, weights, plan and moves captured once and replayed
    step after step: as eagerly, bit for bit."""
    s = Decoder(way, D, Hq, Hkv, P, layout)
    eager = s.run(s.step)
    s = Decoder(way, D, Hq, Hkv, P, layout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    replayed = s.run(graph.replay)
    assert all(base.same_bits(a, b) for a, b in zip(eager, replayed)) and int(s.err.item()) == 0


def test_pools_past_32_bits():
    """Pages behind the 2^31-th element of their pools: as in small ones."""
    D, K, P, counts, lens = 128, 1, 16, [1, 40, 1], [100, 33, 300]
    case = base.wl.mixed_step(41, counts, lens, 4, K, D, P, device=DEV)
    f, _ = base.freqs_of(D)
    far = 2 ** 31 // (P * K * D)
    got = []
    for shift in (0, far):
        kc, vc = (torch.empty((case.num_pages + shift, P, K, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kc[shift:], vc[shift:] = case.k_cache, case.v_cache
        table = base.i32(np.where(case.block_table > 0, case.block_table + shift, 0))
        old, ptr, err = base.i32(lens), base.i32(case.qo_indptr), base.zero()
        slots = case.max_blocks * P
        mass, pos = torch.ones(1, 3, K, slots, device=DEV), torch.zeros(1, 3, K, slots, dtype=torch.int32, device=DEV)
        q = pkv.pkv_rope_append(kc, vc, case.q, case.k_new, case.v_new, table, old, f, append_indptr=ptr, err_flag=err)
        pkv.pkv_attn_mass(kc, q, torch.full((42, 4), 6.0, device=DEV), table, old, case.softmax_scale, mass[0], qo_indptr=ptr,
                          slot_pos=pos[0], err_flag=err)
        now, gone = base.i32(np.array(lens) + counts), base.i32([0, 0, 0])
        moves, num, rows = pkv.pkv_evict_plan(mass, pos, now, gone, base.i32([40, 20, 100]), 1, 4, err_flag=err)
        pkv.pkv_evict_apply(pkv.LayerCaches([kc], [vc]), moves, num, rows, table, now, gone, mass=mass, slot_pos=pos, err_flag=err)
        assert int(err.item()) == 0 and now.tolist() == [40, 20, 100] and int(num.max()) > 0
        got.append([q, kc[shift:].clone(), vc[shift:].clone(), mass, pos])
        del kc, vc
    assert all(base.same_bits(a, b) for a, b in zip(*got))


def test_weights_on_two_streams_at_once():
    """With a workspace each, and a third call behind both."""
    cases = [base.mass_case(s, c, n, 8, 2, 128, 16) for s, c, n in ((42, [600, 1], [100, 900]), (43, [1] * 40, list(range(0, 1600, 40))))]
    want = [base.run_mass(c, z)[1] for c, z in cases]
    calls, streams = [], [torch.cuda.Stream() for _ in cases]
    for (case, z), w in zip(cases, want):
        args = [z.to(DEV), base.i32(case.block_table), base.i32(case.cache_seqlens), base.i32(case.qo_indptr)]
        ws = pkv.mass_workspace(case.batch, case.q.shape[0], case.max_blocks, 8, pkv.cache_desc(case.k_cache), DEV)
        start = torch.rand(w.shape, generator=torch.Generator().manual_seed(1)).to(DEV)
        calls.append((case, args, ws, [start.clone() for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for (case, (z, table, lens, ptr), ws, out), stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                pkv.pkv_attn_mass(case.k_cache, case.q, z, table, lens, case.softmax_scale, out[i], qo_indptr=ptr, workspace=ws,
                                  layout=case.layout)
    torch.cuda.synchronize()
    for (_, _, _, out), w in zip(calls, want):
        assert all(base.same_bits(x.cpu(), w) for x in out)
